"""What the Python binding hands to the library for the operators around the
attention call, with a stand-in for the library (no GPU needed: device addresses
are made up and never used)."""
import threading
import time

import pytest

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

torch = pytest.importorskip("torch")

DEV = 0x7F0000000000


class Fake:
    """Stands for a contiguous tensor on a GPU."""

    def __init__(self, shape, dtype=torch.float16, device=0, base=DEV, contiguous=True):
        self.shape, self.dtype, self.index, self.base, self.contiguous = tuple(shape), dtype, device, base, contiguous
        self.is_cuda = True

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self, i):
        n = 1
        for s in self.shape[i + 1:]:
            n *= s
        return n

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def is_contiguous(self):
        return self.contiguous

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.base


class Library:
    """Answers every call with DS_OK, after `seen` has had its arguments."""

    def __init__(self, seen=lambda name, args: None):
        self.seen = seen

    def __getattr__(self, name):
        def call(*args):
            self.seen(name, args)
            return R.DS_OK
        return call


HQ, HKV, D = 4, 2, 64


def layer_of(n_tokens=5, dtype="fp16", flags=0, max_tokens=8):
    """A RaggedLayer as it is after build(), without its buffers."""
    layer = R.RaggedLayer.__new__(R.RaggedLayer)
    layer.params, layer.stream, layer.rope = R.make_params(HQ, HKV, D, dtype), None, R.ds_rope_table(DEV, 64, D, 1e4)
    layer.meta = R.ds_ragged_meta()
    layer.meta.n_tokens, layer.meta.max_tokens, layer.meta.flags = n_tokens, max_tokens, flags
    return layer


@pytest.fixture
def gpu0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def test_two_threads_append_to_two_pools_through_one_layer(monkeypatch, gpu0):
    """The call runs without the interpreter lock: what one thread passes must not change under it."""
    mine, wrong = threading.local(), []

    def seen(name, args):
        if name == "ds_kv_norm_rotary_append":
            time.sleep(2e-4)  # as a foreign call, lets the other thread run
            pool = args[7]._obj
            if (pool.base, pool.num_blocks) != mine.pool:
                wrong.append((pool.base, mine.pool))

    monkeypatch.setattr(R, "load", lambda: Library(seen))
    layer, norm = layer_of(), R.make_qk_norm(None, None)
    qkv = Fake((5, (HQ + 2 * HKV) * D))

    def work(i):
        pool = Fake((3 + i, 2, HKV, 64, D), base=DEV + (i << 30))
        mine.pool = (pool.base, 3 + i)
        for _ in range(100):
            layer.norm_append(norm, qkv, pool)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, "%d calls saw the other thread's pool" % len(wrong)


WIDTH = (HQ + 2 * HKV) * D


class TestNormAppendTensors:
    """Nothing of another type and nothing short is handed on: the kernel takes 16-bit words at an address."""

    @pytest.fixture
    def calls(self, monkeypatch, gpu0):
        made = []
        monkeypatch.setattr(R, "load", lambda: Library(lambda name, args: made.append(name)))
        return made

    def call(self, calls, refused, norm=None, qkv=None, qkv_out=None, q_out=None, **layer):
        layer = layer_of(**layer)
        norm = norm or R.make_qk_norm(None, None)
        qkv = qkv or Fake((8, WIDTH))
        args = (layer.meta, layer.params, layer.rope, norm, qkv, qkv_out, q_out, R.ds_kv_pool(DEV, 3))
        if refused:
            with pytest.raises(R.DSError):
                R.ds_kv_norm_rotary_append(*args)
        else:
            R.ds_kv_norm_rotary_append(*args)
        assert bool(calls) != refused

    @pytest.mark.parametrize("make", [
        lambda: (Fake((D,), torch.int16), None), lambda: (None, Fake((D,), torch.int16)),
        lambda: (Fake((D,), torch.float16), Fake((D,), torch.bfloat16)), lambda: (Fake((D,), torch.float32), None),
    ])
    def test_weights_of_no_storage_type(self, make):
        with pytest.raises(R.DSError):
            R.make_qk_norm(*make())

    @pytest.mark.parametrize("dtype,other", [("fp16", torch.bfloat16), ("bf16", torch.float16)])
    def test_weights_of_another_type_than_the_layer(self, calls, dtype, other):
        same = torch.bfloat16 if dtype == "bf16" else torch.float16
        for q, k in ((Fake((D,), other), Fake((D,), other)), (Fake((D,), other), None), (None, Fake((D,), other))):
            self.call(calls, True, norm=R.make_qk_norm(q, k), qkv=Fake((8, WIDTH), same), dtype=dtype)
        self.call(calls, False, norm=R.make_qk_norm(Fake((D,), same), None), qkv=Fake((8, WIDTH), same), dtype=dtype)

    @pytest.mark.parametrize("kw", [
        dict(qkv=Fake((4, WIDTH))), dict(qkv=Fake((5, WIDTH - 1))), dict(qkv=Fake((5, WIDTH), torch.bfloat16)),
        dict(qkv=Fake((5, WIDTH), torch.int16)), dict(qkv=Fake((5, WIDTH), torch.float32)),
        dict(qkv_out=Fake((4, WIDTH), base=2 * DEV)), dict(qkv_out=Fake((5, HQ * D), base=2 * DEV)),
        dict(qkv_out=Fake((5, WIDTH), torch.bfloat16, base=2 * DEV)),
        dict(q_out=Fake((4, HQ * D), base=2 * DEV)), dict(q_out=Fake((5, HQ * D), torch.bfloat16, base=2 * DEV)),
        dict(qkv=Fake((5, WIDTH)), flags=R.DS_META_CAPACITY), dict(qkv_out=Fake((7, WIDTH)), flags=R.DS_META_CAPACITY),
        dict(q_out=Fake((7, HQ * D)), flags=R.DS_META_CAPACITY),
    ])
    def test_rows_of_another_type_or_too_few(self, calls, kw):
        self.call(calls, True, **kw)

    @pytest.mark.parametrize("kw", [
        dict(qkv=Fake((5, WIDTH))), dict(qkv=Fake((5, HQ + 2 * HKV, D))), dict(qkv_out=Fake((5, WIDTH)), q_out=Fake((5, HQ, D))),
        dict(qkv_out=Fake((8, WIDTH)), q_out=Fake((8, HQ * D)), flags=R.DS_META_CAPACITY),
        dict(qkv=Fake((1, WIDTH)), n_tokens=0),
    ])
    def test_rows_that_fit(self, calls, kw):
        self.call(calls, False, **kw)

    @pytest.mark.parametrize("pool,refused", [
        (Fake((3, 2, HKV, 64, D)), False), (Fake((3, 2 * HKV * 64 * D)), False), (Fake((0, 2, HKV, 64, D)), False),
        (Fake((3, 2, HKV, 64, D), torch.bfloat16), True), (Fake((3, 2, HKV - 1, 64, D)), True),
        (Fake((3, 2, HKV, 32, D)), True), (Fake((3, 2, HKV, 64, D), contiguous=False), True),
    ])
    def test_pool_of_another_layer(self, calls, pool, refused):
        layer, norm, qkv = layer_of(), R.make_qk_norm(None, None), Fake((5, WIDTH))
        if refused:
            with pytest.raises(R.DSError):
                layer.norm_append(norm, qkv, pool)
        else:
            layer.norm_append(norm, qkv, pool)
        assert bool(calls) != refused


class TestDevices:
    """The library launches on the current device (0 here): whatever lies on another one is refused."""

    @pytest.fixture(autouse=True)
    def library(self, monkeypatch, gpu0):
        self.calls = []
        monkeypatch.setattr(R, "load", lambda: Library(lambda name, args: self.calls.append(name)))

    def check(self, names, call):
        call({})
        assert len(self.calls) == 1
        for name in names:
            with pytest.raises(R.DSError, match="device"):
                call({name: 1})
        assert len(self.calls) == 1

    def test_norm_append(self):
        def call(where):
            f = lambda name, *shape: Fake(shape, device=where.get(name, 0))  # noqa: E731
            norm = R.make_qk_norm(f("q_weight", D), f("k_weight", D))
            layer_of().norm_append(norm, f("qkv", 5, WIDTH), f("pool", 3, 2, HKV, 64, D), f("qkv_out", 5, WIDTH), f("q_out", 5, HQ * D))
        self.check(["q_weight", "k_weight", "qkv", "pool", "qkv_out", "q_out"], call)
        with pytest.raises(R.DSError, match="device"):  # all weights together
            layer_of().norm_append(R.make_qk_norm(Fake((D,), device=1), None), Fake((5, WIDTH)), Fake((3, 2, HKV, 64, D)))

    def test_lora(self):
        def call(where):
            f = lambda name, *shape, dtype=torch.float16: Fake(shape, dtype, where.get(name, 0))  # noqa: E731
            plan = R.ds_lora_plan()
            plan.n_tokens, plan.device = 5, where.get("plan", 0)
            lora = R.make_lora(f("a", 2, 8, 64), f("b", 2, 96, 8), f("scale", 2, dtype=torch.float32))
            R.ds_ragged_lora(plan, lora, f("x", 5, 64), f("base", 5, 96), f("out", 5, 96))
        self.check(["a", "b", "scale", "x", "base", "out", "plan"], call)
        plan = R.ds_lora_plan()
        plan.n_tokens = 5
        lora = R.make_lora(Fake((2, 8, 64), device=1), Fake((2, 96, 8), device=1))
        with pytest.raises(R.DSError, match="device 1"):
            R.ds_ragged_lora(plan, lora, Fake((5, 64)), Fake((5, 96)), Fake((5, 96)))

    def test_sample(self):
        def call(where):
            f = lambda name, *shape, dtype=torch.float32: Fake(shape, dtype, where.get(name, 0))  # noqa: E731
            meta = R.ds_ragged_meta()
            meta.n_seqs = 4
            i32 = torch.int32
            s = R.make_sampler(f("uniforms", 4), f("temperature", 4), f("top_k", 4, dtype=i32), f("top_p", 4), f("min_p", 4))
            R.ds_ragged_sample(meta, f("logits", 4, 99), s, f("tokens", 4, dtype=i32), f("logprobs", 4))
        self.check(["uniforms", "temperature", "top_k", "top_p", "min_p", "logits", "tokens", "logprobs"], call)
        meta = R.ds_ragged_meta()
        meta.n_seqs = 4
        with pytest.raises(R.DSError, match="device 1"):
            R.ds_ragged_sample(meta, Fake((4, 99)), R.make_sampler(Fake((4,), torch.float32, 1)), Fake((4,), torch.int32))

"""Refusals of the operators around the attention call, found on the host before
anything is launched (no GPU needed: device addresses are made up and never used)."""
import ctypes

import numpy as np
import pytest

from ragged_blocked_kv_raggedbatch_gb300 import build as B
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

DEV = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    B.build()
    return R.load()


def packed(seqs, hq=4, hkv=2, d=64, flags=0):
    """(params, meta, staging) of a batch packed against a made-up device buffer."""
    wl = W.make_custom(seqs, hq, hkv, d, dtype="fp16")
    params = R.params_for(wl)
    nb = int(wl.blocks_needed().sum()) if wl.n_seqs else 0
    dev, stg = R.ds_meta_buffer_sizes(max(wl.n_seqs, 1), max(wl.n_tokens, 1), max(nb, 1), params)
    stage = np.zeros(stg // 4 + 4, np.int32)
    meta = R.ds_ragged_meta()
    meta.device_buf, meta.device_bytes = DEV, dev
    meta.host_staging, meta.staging_bytes = stage.ctypes.data, stg
    meta.max_seqs, meta.max_tokens, meta.max_blocks = max(wl.n_seqs, 1), max(wl.n_tokens, 1), max(nb, 1)
    meta.flags = flags
    assert R.ds_ragged_meta_pack(R.SeqDescs.of(wl), params, wl.num_blocks, meta) == R.DS_OK
    return params, meta, stage, wl


class TestNormAppend:
    def call(self, lib, **kw):
        params, meta, stage, wl = packed(kw.pop("seqs", [(3, 5), (64, 1)]))
        a = dict(norm=R.ds_qk_norm(DEV, DEV, 0, 1e-6), qkv=DEV, qkv_out=None, q_out=None,
                 rope=R.ds_rope_table(DEV, 4096, params.head_dim, params.rope_theta),
                 pool=R.ds_kv_pool(DEV, wl.num_blocks), meta=meta, params=params)
        a.update(kw)
        ref = R._ref
        return lib.ds_kv_norm_rotary_append(ref(a["meta"]), ref(a["params"]), ref(a["rope"]), ref(a["norm"]), a["qkv"],
                                            a["qkv_out"], a["q_out"], ref(a["pool"]), None)

    @pytest.mark.parametrize("kw", [
        dict(norm=None), dict(qkv=None), dict(qkv=DEV + 2), dict(qkv_out=DEV + (1 << 30) + 8), dict(q_out=DEV + (1 << 30) + 8),
        dict(norm=R.ds_qk_norm(DEV + 2, DEV, 0, 1e-6)), dict(norm=R.ds_qk_norm(DEV, DEV + 8, 0, 1e-6)),
        dict(norm=R.ds_qk_norm(DEV, DEV, 0, 0.0)), dict(norm=R.ds_qk_norm(DEV, DEV, 0, -1.0)),
        dict(norm=R.ds_qk_norm(DEV, DEV, 0, float("nan"))), dict(norm=R.ds_qk_norm(DEV, DEV, 0, float("inf"))),
        dict(norm=R.ds_qk_norm(DEV, DEV, 2, 1e-6)),
        dict(qkv_out=DEV + 512), dict(q_out=DEV), dict(qkv_out=DEV + (1 << 30), q_out=DEV + (1 << 30) + 512),
        dict(rope=None), dict(pool=None), dict(pool=R.ds_kv_pool(DEV, 1)), dict(meta=None), dict(params=None),
        dict(rope=R.ds_rope_table(DEV, 4096, 128, 1e4)),
    ])
    def test_refuses(self, lib, kw):
        assert self.call(lib, **kw) == R.DS_ERR_INVALID_ARG
        assert lib.ds_last_error()

    def test_refuses_positions_beyond_the_table(self, lib):
        assert self.call(lib, rope=R.ds_rope_table(DEV, 64, 64, 1e4)) == R.DS_ERR_CAPACITY

    def test_empty_batch_is_no_work(self, lib):
        assert self.call(lib, seqs=[], rope=None, pool=None, qkv=None) == R.DS_OK


class TestSample:
    def call(self, lib, **kw):
        params, meta, stage, wl = packed(kw.pop("seqs", [(3, 5), (64, 1)]))
        a = dict(meta=meta, logits=DEV, dtype=R.DS_FP32, vocab=1000, stride=1000, sampler=R.ds_sampler(DEV), tokens=DEV, logprobs=None)
        a.update(kw)
        return lib.ds_ragged_sample(R._ref(a["meta"]), a["logits"], a["dtype"], a["vocab"], a["stride"], R._ref(a["sampler"]),
                                    a["tokens"], a["logprobs"], None)

    @pytest.mark.parametrize("kw", [
        dict(meta=None), dict(meta=R.ds_ragged_meta()), dict(logits=None), dict(logits=DEV + 2), dict(logits=DEV + 1, dtype=R.DS_BF16),
        dict(vocab=0), dict(vocab=-3), dict(stride=999), dict(sampler=None), dict(sampler=R.ds_sampler()),
        dict(sampler=R.ds_sampler(DEV + 2)), dict(sampler=R.ds_sampler(DEV, DEV + 1)), dict(sampler=R.ds_sampler(DEV, None, DEV + 2)),
        dict(sampler=R.ds_sampler(DEV, None, None, DEV + 2)), dict(sampler=R.ds_sampler(DEV, None, None, None, DEV + 3)),
        dict(tokens=None), dict(tokens=DEV + 2), dict(logprobs=DEV + 2),
    ])
    def test_refuses(self, lib, kw):
        assert self.call(lib, **kw) == R.DS_ERR_INVALID_ARG
        assert lib.ds_last_error()

    def test_unsupported(self, lib):
        assert self.call(lib, dtype=3) == R.DS_ERR_UNSUPPORTED
        assert self.call(lib, dtype=-1) == R.DS_ERR_UNSUPPORTED
        assert self.call(lib, vocab=262145, stride=262145) == R.DS_ERR_UNSUPPORTED

    def test_empty_batch_is_no_work(self, lib):
        assert self.call(lib, seqs=[], logits=None, tokens=None) == R.DS_OK

    def test_binding_refuses_host_tensors(self):
        torch = pytest.importorskip("torch")
        with pytest.raises(R.DSError):
            R.make_sampler(torch.zeros(2))
        with pytest.raises(R.DSError):
            R.make_sampler(None)
        with pytest.raises(R.DSError):
            R.make_qk_norm(torch.zeros(64), None)
        with pytest.raises(R.DSError):
            R.make_lora(torch.zeros(1, 8, 64), torch.zeros(1, 64, 8))
        params, meta, stage, wl = packed([(3, 5)])
        with pytest.raises(R.DSError):
            R.ds_kv_norm_rotary_append(meta, params, R.ds_rope_table(DEV, 64, 64, 1e4), R.make_qk_norm(None, None),
                                       torch.zeros(5, 512, dtype=torch.float16), None, None, R.ds_kv_pool(DEV, wl.num_blocks))
        with pytest.raises(R.DSError):
            R.ds_ragged_sample(meta, torch.zeros(1, 8), R.ds_sampler(DEV), torch.zeros(1, dtype=torch.int32))

    def test_binding_refuses_tensors_of_another_device(self, monkeypatch):
        torch = pytest.importorskip("torch")
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

        class Elsewhere:  # stands for a tensor on device 1
            is_cuda, dtype, shape = True, torch.float16, (5, 512)
            is_contiguous = lambda self: True  # noqa: E731
            get_device = lambda self: 1  # noqa: E731
            data_ptr = lambda self: DEV  # noqa: E731
            stride = lambda self, i: (512, 1)[i]  # noqa: E731

        t = Elsewhere()
        params, meta, stage, wl = packed([(3, 5)])
        with pytest.raises(R.DSError, match="device 1"):
            R.ds_kv_norm_rotary_append(meta, params, R.ds_rope_table(DEV, 64, 64, 1e4), R.make_qk_norm(None, None), t, None, None,
                                       R.ds_kv_pool(DEV, wl.num_blocks))
        with pytest.raises(R.DSError, match="device 1"):
            R.ds_ragged_sample(meta, t, R.ds_sampler(DEV), None)
        plan = Plan()
        assert plan.pack([5], [0], 1) == R.DS_OK
        lora = R.ds_lora_weights(DEV, DEV, None, 1, 16, 512, 512, R.DS_FP16)
        lora.tensors = (t,)
        with pytest.raises(R.DSError, match="device 1"):
            R.ds_ragged_lora(plan.p, lora, t, t, t)


class Plan:
    def __init__(self, max_seqs=8, max_tokens=500, flags=0):
        dev, stg = ctypes.c_size_t(0), ctypes.c_size_t(0)
        assert R.load().ds_lora_plan_size(max_seqs, max_tokens, ctypes.byref(dev), ctypes.byref(stg)) == R.DS_OK
        self.stage = np.zeros(stg.value // 4 + 4, np.int32)
        self.stage[-4:] = 123456
        at = self.stage.ctypes.data
        self.stage_at = at + (-at) % 16
        self.p = R.ds_lora_plan(DEV, dev.value, self.stage_at, stg.value, max_seqs, max_tokens, flags)

    def pack(self, new, which, n_adapters):
        new, which = np.array(new, np.int32), np.array(which, np.int32)
        return R.load().ds_lora_plan_pack(new.ctypes.data, which.ctypes.data, len(new), n_adapters, R._ref(self.p))

    def image(self):
        w = np.array((ctypes.c_int32 * (self.p.used_bytes // 4)).from_address(self.stage_at))
        at = lambda ptr: (ptr - DEV) // 4  # noqa: E731
        s, l = self.p.n_small_tiles, self.p.n_large_tiles
        return (w[:4], w[at(self.p.order):at(self.p.small_tiles)], w[at(self.p.small_tiles):][:4 * s].reshape(-1, 4),
                w[at(self.p.large_tiles):][:12 * l].reshape(-1, 12))


class TestLora:
    @pytest.mark.parametrize("flags", [0, R.DS_META_CAPACITY])
    @pytest.mark.parametrize("seed", range(12))
    def test_plan_covers_every_token_once(self, lib, seed, flags):
        r = np.random.RandomState(seed)
        n, na = r.randint(1, 40), r.randint(1, 9)
        new = np.where(r.rand(n) < 0.5, 1, r.randint(1, 200, n))
        which = r.randint(-1, na, n)
        plan = Plan(n, int(new.sum()) + seed, flags)
        assert plan.pack(new, which, na) == R.DS_OK
        assert plan.p.used_bytes <= plan.p.device_bytes and (plan.stage[-4:] == 123456).all()
        head, order, small, large = plan.image()
        assert list(head[:3]) == [len(small), len(large), new.sum()]
        token = np.repeat(which, new)
        done = np.zeros(new.sum(), int)
        for a, first, count, _ in small:
            assert 1 <= count <= 16
            mine = order[first:first + count]
            assert (token[mine] == a).all()
            done[mine] += 1
        for tile in large:
            assert 1 <= tile[2] <= 32
            for first, count in tile[1:9].reshape(4, 2):
                assert 0 <= count <= 32 and (token[first:first + count] == tile[0]).all()
                done[first:first + count] += 1
        assert (done == 1).all()

    @pytest.mark.parametrize("new,which,na,status", [
        ([1, 0], [0, 0], 1, R.DS_ERR_INVALID_ARG), ([1, -2], [0, 0], 1, R.DS_ERR_INVALID_ARG),
        ([1], [1], 1, R.DS_ERR_INVALID_ARG), ([1], [-2], 1, R.DS_ERR_INVALID_ARG), ([1], [0], 0, R.DS_ERR_INVALID_ARG),
        ([1], [0], -1, R.DS_ERR_INVALID_ARG), ([1] * 9, [0] * 9, 1, R.DS_ERR_CAPACITY), ([501], [0], 1, R.DS_ERR_CAPACITY),
        ([2 ** 31 - 1, 2 ** 31 - 1], [0, 0], 1, R.DS_ERR_CAPACITY),
    ])
    def test_pack_refuses(self, lib, new, which, na, status):
        assert Plan().pack(new, which, na) == status and lib.ds_last_error()

    def test_pack_refuses_buffers(self, lib):
        one = np.zeros(1, np.int32)
        for change in (dict(device_buf=None), dict(device_buf=DEV + 16), dict(host_staging=None), dict(flags=2)):
            plan = Plan()
            for k, v in change.items():
                setattr(plan.p, k, v)
            assert plan.pack([1], [0], 1) == R.DS_ERR_INVALID_ARG
        plan = Plan()
        plan.p.device_bytes -= 256
        assert plan.pack([1], [0], 1) == R.DS_ERR_WORKSPACE
        assert lib.ds_lora_plan_pack(None, one.ctypes.data, 1, 1, R._ref(Plan().p)) == R.DS_ERR_INVALID_ARG
        assert lib.ds_lora_plan_pack(one.ctypes.data, one.ctypes.data, 1, 1, None) == R.DS_ERR_INVALID_ARG
        assert lib.ds_lora_plan_size(-1, 4, one.ctypes.data, one.ctypes.data) == R.DS_ERR_INVALID_ARG
        assert lib.ds_lora_plan_size(1, 4, None, None) == R.DS_ERR_INVALID_ARG

    def call(self, lib, **kw):
        plan = Plan()
        assert plan.pack(kw.pop("new", [1, 20]), kw.pop("which", [0, 1]), 2) == R.DS_OK
        w = dict(a=DEV, b=DEV, scale=DEV, n_adapters=2, rank=16, in_dim=64, out_dim=128, dtype=R.DS_BF16)
        far = 1 << 30
        c = dict(plan=plan.p, x=DEV, xs=64, base=DEV + far, bs=128, out=DEV + 2 * far, os=128, lora=True)
        for k, v in kw.items():
            (w if k in w else c)[k] = v
        lora = R._ref(R.ds_lora_weights(*w.values())) if c["lora"] else None
        return lib.ds_ragged_lora(R._ref(c["plan"]), lora, c["x"], c["xs"], c["base"], c["bs"], c["out"], c["os"], None)

    @pytest.mark.parametrize("kw", [
        dict(plan=None), dict(plan=R.ds_lora_plan()), dict(lora=None), dict(n_adapters=3), dict(a=None), dict(b=DEV + 8), dict(scale=DEV + 2),
        dict(x=None), dict(base=None), dict(out=None), dict(x=DEV + 8), dict(base=DEV + 2), dict(out=DEV + 4),
        dict(xs=56), dict(bs=120), dict(os=0), dict(xs=68), dict(bs=129), dict(os=132),
        dict(out=DEV), dict(out=DEV + 64 * 2 * 20), dict(out=DEV + (1 << 30) + 256), dict(out=DEV + (1 << 30), os=256),
    ])
    def test_refuses(self, lib, kw):
        assert self.call(lib, **kw) == R.DS_ERR_INVALID_ARG and lib.ds_last_error()

    @pytest.mark.parametrize("kw", [dict(rank=0), dict(rank=12), dict(rank=136), dict(in_dim=60), dict(out_dim=0), dict(dtype=R.DS_FP32)])
    def test_unsupported(self, lib, kw):
        assert self.call(lib, **kw) == R.DS_ERR_UNSUPPORTED

    def test_error_word_refuses(self, lib):
        v = ctypes.c_int32(0)
        assert lib.ds_lora_get_device_error(None, ctypes.byref(v), None) == R.DS_ERR_INVALID_ARG
        assert lib.ds_lora_get_device_error(R._ref(R.ds_lora_plan()), ctypes.byref(v), None) == R.DS_ERR_INVALID_ARG
        plan = Plan()
        assert plan.pack([1], [0], 1) == R.DS_OK
        assert lib.ds_lora_get_device_error(R._ref(plan.p), None, None) == R.DS_ERR_INVALID_ARG

    def test_empty_batch_is_no_work(self, lib):
        assert self.call(lib, new=[], which=[], x=None, base=None, out=None) == R.DS_OK

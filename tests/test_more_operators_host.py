"""Refusals of the calls on the 8-bit pool and of the rules on logits, found on the host
before anything is launched, and what the binding hands on (no GPU needed: device
addresses are made up and never used)."""
import pytest

import test_operator_binding as OB
import test_operators_host as H
from ragged_blocked_kv_raggedbatch_gb300 import build as B
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

torch = pytest.importorskip("torch")
DEV, FAR = H.DEV, 1 << 30
Fake = OB.Fake


@pytest.fixture(scope="module")
def lib():
    B.build()
    return R.load()


@pytest.fixture
def gpu0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


class TestPool:
    def call(self, lib, name, flags=0, **kw):
        params, meta, stage, wl = H.packed(kw.pop("seqs", [(3, 5), (64, 1)]), flags=flags)
        a = dict(meta=meta, params=params, rope=R.ds_rope_table(DEV, 4096, params.head_dim, params.rope_theta), qkv=DEV,
                 pool=R.ds_kv8_pool(DEV, DEV + FAR, wl.num_blocks), out=DEV + 2 * FAR, ws=DEV + 3 * FAR, ws_bytes=1 << 28)
        a.update(kw)
        first = [R._ref(a["meta"]), R._ref(a["params"]), R._ref(a["rope"]), a["qkv"], R._ref(a["pool"])]
        if name == "append":
            return lib.ds_kv8_rotary_append(*first, None)
        return lib.ds_kv8_blocked_attention(*first, a["out"], a["ws"], a["ws_bytes"], None)

    @pytest.mark.parametrize("name", ["append", "attention"])
    @pytest.mark.parametrize("kw", [
        dict(meta=None), dict(meta=R.ds_ragged_meta()), dict(params=None), dict(rope=None), dict(rope=R.ds_rope_table(DEV, 4096, 128, 1e4)),
        dict(rope=R.ds_rope_table(DEV, 4096, 64, 5e5)), dict(qkv=None), dict(qkv=DEV + 8), dict(pool=None),
        dict(pool=R.ds_kv8_pool(None, DEV, 3)), dict(pool=R.ds_kv8_pool(DEV, None, 3)), dict(pool=R.ds_kv8_pool(DEV + 8, DEV, 3)),
        dict(pool=R.ds_kv8_pool(DEV, DEV + 2, 3)), dict(pool=R.ds_kv8_pool(DEV, DEV, 1)),
    ])
    def test_refuses(self, lib, name, kw):
        assert self.call(lib, name, **kw) == R.DS_ERR_INVALID_ARG and lib.ds_last_error()

    @pytest.mark.parametrize("kw,status", [
        (dict(out=None), R.DS_ERR_INVALID_ARG), (dict(out=DEV + 8), R.DS_ERR_INVALID_ARG), (dict(ws=None), R.DS_ERR_INVALID_ARG),
        (dict(ws=DEV + 128), R.DS_ERR_INVALID_ARG), (dict(ws_bytes=16), R.DS_ERR_WORKSPACE),
    ])
    def test_attention_refuses(self, lib, kw, status):
        assert self.call(lib, "attention", **kw) == status and lib.ds_last_error()

    def test_workspace_of_the_capacities(self, lib):
        """A captured call may be replayed for any batch: the workspace is for the capacities, also without decode rows."""
        assert self.call(lib, "attention", flags=R.DS_META_CAPACITY, seqs=[(3, 5)], ws_bytes=16) == R.DS_ERR_WORKSPACE

    @pytest.mark.parametrize("name", ["append", "attention"])
    def test_positions_beyond_the_table(self, lib, name):
        assert self.call(lib, name, rope=R.ds_rope_table(DEV, 64, 64, 1e4)) == R.DS_ERR_CAPACITY

    @pytest.mark.parametrize("name", ["append", "attention"])
    def test_unsupported_shapes(self, lib, name):
        for bad in (R.make_params(6, 2, 64, "fp16"), R.make_params(4, 2, 96, "fp16"), R.make_params(4, 2, 64, R.DS_FP32),
                    R.make_params(4, 2, 64, "fp16", block_size=32)):
            assert self.call(lib, name, params=bad) == R.DS_ERR_UNSUPPORTED

    @pytest.mark.parametrize("name", ["append", "attention"])
    def test_empty_batch_is_no_work(self, lib, name):
        assert self.call(lib, name, seqs=[], rope=None, pool=None, qkv=None, out=None, ws=None) == R.DS_OK


class TestRules:
    RULES = dict(history=DEV, history_stride=100, history_len=DEV, prompt_len=DEV, repetition=DEV, frequency=DEV, presence=DEV,
                 bias_ids=DEV, bias_values=DEV, bias_stride=5, bias_len=DEV, mask=DEV, mask_stride=32, n_masks=2, mask_row=DEV)

    def call(self, lib, flags=0, **kw):
        params, meta, stage, wl = H.packed(kw.pop("seqs", [(3, 5), (64, 1)]), flags=flags)
        rules = dict(self.RULES)
        a = dict(meta=meta, logits=DEV, dtype=R.DS_BF16, vocab=1000, stride=1000, rules=True, out=DEV + FAR, out_stride=1000)
        for k, v in kw.items():
            (rules if k in rules else a)[k] = v
        r = R._ref(R.ds_logit_rules(*rules.values())) if a["rules"] else None
        return lib.ds_ragged_adjust_logits(R._ref(a["meta"]), a["logits"], a["dtype"], a["vocab"], a["stride"], r, a["out"],
                                           a["out_stride"], None)

    @pytest.mark.parametrize("kw", [
        dict(meta=None), dict(meta=R.ds_ragged_meta()), dict(rules=None), dict(logits=None), dict(out=None), dict(logits=DEV + 1),
        dict(out=DEV + FAR + 1), dict(dtype=R.DS_FP32, logits=DEV + 2), dict(vocab=0), dict(vocab=-1), dict(stride=999), dict(out_stride=999),
        dict(history=None), dict(history_len=None), dict(history_stride=-1), dict(bias_ids=None), dict(bias_values=None), dict(bias_stride=-1),
        dict(mask_stride=31), dict(n_masks=-1), dict(n_masks=1, mask_row=None),
        dict(out=DEV, out_stride=1001), dict(out=DEV + 2), dict(out=DEV + 1999 * 2), dict(out=DEV - 1999 * 2),
    ] + [{k: DEV + 2} for k in RULES if not k.endswith("stride") and k != "n_masks"])
    def test_refuses(self, lib, kw):
        assert self.call(lib, **kw) == R.DS_ERR_INVALID_ARG and lib.ds_last_error()

    @pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(history_stride=1 << 19), dict(bias_stride=2047),
                                    dict(vocab=(1 << 28) + 1, stride=1 << 29, out_stride=1 << 29, mask_stride=1 << 24)])
    def test_unsupported(self, lib, kw):
        assert self.call(lib, **kw) == R.DS_ERR_UNSUPPORTED and lib.ds_last_error()

    @pytest.mark.parametrize("kw", [dict(out=DEV + 6000 * 2), dict(out=DEV - 6000 * 2)])
    def test_rows_of_the_capacity(self, lib, kw):
        """Two sequences in buffers of eight: rows that only a later batch reaches may not meet either."""
        params, meta, stage, wl = H.packed([(3, 5), (64, 1)])
        meta.flags, meta.max_seqs = R.DS_META_CAPACITY, 8
        assert self.call(lib, meta=meta, **kw) == R.DS_ERR_INVALID_ARG
        assert b"overlaps" in lib.ds_last_error()

    def test_empty_batch_is_no_work(self, lib):
        assert self.call(lib, seqs=[], logits=None, out=None) == R.DS_OK


class TestBinding:
    """Nothing of another type, shape or device and nothing short is handed on."""

    @pytest.fixture
    def calls(self, monkeypatch, gpu0):
        made = []
        monkeypatch.setattr(R, "load", lambda: OB.Library(lambda name, args: made.append((name, args))))
        return made

    def pool(self, blocks=3, heads=OB.HKV, d=OB.D, device=0, dtype=None, **kw):
        return R.make_kv8_pool(Fake((blocks, 2, heads, 64, d), dtype or torch.uint8, device, **kw),
                               Fake((blocks, 2, heads), torch.float32, device))

    def test_pool(self, gpu0):
        assert self.pool().num_blocks == 3 and self.pool(dtype=torch.float8_e4m3fn).num_blocks == 3
        good, scales = Fake((3, 2, 2, 64, 64), torch.uint8), Fake((3, 2, 2), torch.float32)
        for c, s in ((Fake((3, 2, 2, 64, 64), torch.float16), scales), (good, Fake((3, 2, 2), torch.float64)), (good, Fake((3, 2, 4), torch.float32)),
                     (Fake((3, 1, 2, 64, 64), torch.uint8), scales), (Fake((6, 2, 64, 64), torch.uint8), scales),
                     (Fake((3, 2, 2, 64, 64), torch.uint8, contiguous=False), scales), (good, Fake((3, 2, 2), torch.float32, contiguous=False)),
                     (good, Fake((3, 2, 2), torch.float32, 1)), (torch.zeros(3, 2, 2, 64, 64, dtype=torch.uint8), torch.zeros(3, 2, 2))):
            with pytest.raises(R.DSError):
                R.make_kv8_pool(c, s)

    def test_calls_on_the_pool(self, calls):
        layer, width = OB.layer_of(), OB.WIDTH
        layer.workspace = Fake((4096,), torch.uint8)
        qkv, out = Fake((5, width)), Fake((5, OB.HQ * OB.D))
        layer.append8(qkv, self.pool())
        layer.attention8(qkv, self.pool(), out)
        assert [c[0] for c in calls] == ["ds_kv8_rotary_append", "ds_kv8_blocked_attention"] and calls[1][1][7] == 4096
        done = len(calls)
        for q in (Fake((4, width)), Fake((5, width), torch.bfloat16), Fake((5, width), device=1), Fake((5, width), contiguous=False)):
            with pytest.raises(R.DSError):
                layer.append8(q, self.pool())
            with pytest.raises(R.DSError):
                layer.attention8(q, self.pool(), out)
        for p in (self.pool(heads=4), self.pool(d=128), self.pool(device=1)):
            with pytest.raises(R.DSError):
                layer.append8(qkv, p)
            with pytest.raises(R.DSError):
                layer.attention8(qkv, p, out)
        for o in (Fake((4, OB.HQ * OB.D)), Fake((5, OB.HQ * OB.D), torch.bfloat16), Fake((5, OB.HQ * OB.D), device=1)):
            with pytest.raises(R.DSError):
                layer.attention8(qkv, self.pool(), o)
        layer.workspace = Fake((4096,), torch.uint8, device=1)
        with pytest.raises(R.DSError):
            layer.attention8(qkv, self.pool(), out)
        cap = OB.layer_of(flags=R.DS_META_CAPACITY, max_tokens=8)
        with pytest.raises(R.DSError):
            cap.append8(qkv, self.pool())  # rows for the capacities
        cap.append8(Fake((8, width)), self.pool())
        assert len(calls) == done + 1

    def rules(self, rows=3, **kw):
        i, f = torch.int32, torch.float32
        a = dict(history=Fake((rows, 9), i), history_len=Fake((rows,), i), prompt_len=Fake((rows,), i), repetition=Fake((rows,), f),
                 frequency=Fake((rows,), f), presence=Fake((rows,), f), bias_ids=Fake((rows, 4), i), bias_values=Fake((rows, 4), f),
                 bias_len=Fake((rows,), i), mask=Fake((2, 4), i), mask_row=Fake((rows,), i))
        a.update(kw)
        return R.make_logit_rules(**a)

    def test_rules(self, gpu0):
        r = self.rules()
        assert (r.history_stride, r.bias_stride, r.mask_stride, r.n_masks, r.rows) == (9, 4, 4, 2, 3)
        assert R.make_logit_rules().rows is None
        f = torch.float32
        for kw in (dict(history=Fake((3, 9), torch.int64)), dict(history=None), dict(history_len=None), dict(history=Fake((27,), torch.int32)),
                   dict(repetition=Fake((3,), torch.float16)), dict(bias_ids=None), dict(bias_values=None), dict(bias_values=Fake((3, 5), f)),
                   dict(bias_ids=None, bias_values=None), dict(mask=None), dict(mask=Fake((2, 4), torch.int32, contiguous=False)),
                   dict(presence=Fake((3,), f, device=1)), dict(mask_row=torch.zeros(3, dtype=torch.int32))):
            with pytest.raises(R.DSError):
                self.rules(**kw)

    def test_adjust(self, calls):
        meta = OB.layer_of().meta
        meta.n_seqs, meta.max_seqs = 3, 4
        x, y = Fake((3, 100), torch.bfloat16), Fake((3, 100), torch.bfloat16, base=DEV + FAR)
        R.ds_ragged_adjust_logits(meta, x, self.rules(), y)
        R.ds_ragged_adjust_logits(meta, x, self.rules(), x)
        R.ds_ragged_adjust_logits(meta, x, R.make_logit_rules(), y)
        assert len(calls) == 3 and calls[0][1][2:5] == (R.DS_BF16, 100, 100)
        for a, b in ((Fake((3, 100), torch.int32), y), (x, Fake((3, 100), torch.float16)), (x, Fake((3, 99), torch.bfloat16)),
                     (Fake((2, 100), torch.bfloat16), y), (x, Fake((2, 100), torch.bfloat16)), (Fake((3, 100), torch.bfloat16, device=1), y),
                     (x, Fake((3, 100), torch.bfloat16, device=1))):
            with pytest.raises(R.DSError):
                R.ds_ragged_adjust_logits(meta, a, self.rules(), b)
        with pytest.raises(R.DSError):
            R.ds_ragged_adjust_logits(meta, x, self.rules(2), y)
        meta.flags = R.DS_META_CAPACITY  # rows and rules for max_seqs
        with pytest.raises(R.DSError):
            R.ds_ragged_adjust_logits(meta, x, self.rules(4), y)
        with pytest.raises(R.DSError):
            R.ds_ragged_adjust_logits(meta, Fake((4, 100), torch.bfloat16), self.rules(), Fake((4, 100), torch.bfloat16))
        assert len(calls) == 3

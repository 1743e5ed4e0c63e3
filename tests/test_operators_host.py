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

"""Buffers that meet, found on the host before anything is launched (no GPU needed:
device addresses are made up and never used).  With DS_META_CAPACITY a call may be
captured for a small batch and replayed for any up to the capacities: what counts
is the rows of the capacities."""
import pytest

import test_operators_host as H
from ragged_blocked_kv_raggedbatch_gb300 import build as B
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

DEV = H.DEV


@pytest.fixture(scope="module")
def lib():
    B.build()
    return R.load()




def lora(lib, flags, new, which, **kw):
    plan = H.Plan(8, 500, flags)
    assert plan.pack(new, which, 2) == R.DS_OK
    w = R.ds_lora_weights(DEV, DEV, DEV, 2, 16, 64, 128, R.DS_BF16)
    far = 1 << 30
    c = dict(x=DEV, base=DEV + far, out=DEV + 2 * far)
    c.update(kw)
    return lib.ds_ragged_lora(R._ref(plan.p), R._ref(w), c["x"], 64, c["base"], 128, c["out"], 128, None)


@pytest.mark.parametrize("new,which", [([1, 20], [0, 1]), ([], []), ([1], [-1])])
@pytest.mark.parametrize("where", ["x", "base"])
def test_lora_rows_of_the_capacity(lib, new, which, where):
    """out begins inside x's or base's last row of max_tokens = 500."""
    last = dict(x=DEV + 499 * 64 * 2, base=DEV + (1 << 30) + 499 * 128 * 2)[where]
    assert lora(lib, R.DS_META_CAPACITY, new, which, out=last) == R.DS_ERR_INVALID_ARG
    assert b"overlaps " + where.encode() in lib.ds_last_error()
    # and out's last row is the one that meets them
    before = dict(x=DEV, base=DEV + (1 << 30))[where] - 499 * 128 * 2
    assert lora(lib, R.DS_META_CAPACITY, new, which, out=before) == R.DS_ERR_INVALID_ARG


def norm_append(lib, flags, max_tokens, **kw):
    params, meta, stage, wl = H.packed([(3, 5), (64, 1)])
    meta.flags, meta.max_tokens = flags, max_tokens
    c = dict(qkv=DEV, qkv_out=None, q_out=None, blocks=1)  # a pool of one block is refused last
    c.update(kw)
    rope = R.ds_rope_table(DEV, 4096, params.head_dim, params.rope_theta)
    return lib.ds_kv_norm_rotary_append(R._ref(meta), R._ref(params), R._ref(rope), R._ref(R.ds_qk_norm(DEV, DEV, 0, 1e-6)), c["qkv"],
                                      c["qkv_out"], c["q_out"], R._ref(R.ds_kv_pool(DEV + (8 << 30), wl.num_blocks)), None)


@pytest.mark.parametrize("kw", [
    dict(qkv_out=DEV + 99 * 512 * 2), dict(qkv_out=DEV - 99 * 512 * 2), dict(q_out=DEV + 99 * 512 * 2), dict(q_out=DEV - 99 * 256 * 2),
    dict(qkv_out=DEV + (1 << 30), q_out=DEV + (1 << 30) + 99 * 512 * 2),
])
def test_norm_append_rows_of_the_capacity(lib, kw):
    """512 columns of qkv, 256 of q_out, a batch of 6 tokens in buffers of max_tokens = 100."""
    assert norm_append(lib, R.DS_META_CAPACITY, 100, **kw) == R.DS_ERR_INVALID_ARG
    assert b"overlaps" in lib.ds_last_error()

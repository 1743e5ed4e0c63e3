"""GPU: attention over 8-bit pools whose tiles' scales lie far apart: every dimension of a result holds, also one that the
tile of the largest scale has nothing in.  The bound is derived in kv8_bounds."""
import numpy as np
import pytest
import torch

import kv8_bounds as B
import kv8_formula as K
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HEADS = [(4, 2, 64), (8, 1, 128), (3, 3, 64), (2, 2, 128)]


def batch(seqs, heads, dtype, seed=3):
    """A batch with a pool of scale 1 whose codes are e4m3 numbers of normal values, and queries that leave weights of 2^-6 to 1."""
    wl = W.make_custom(seqs, *heads, dtype=dtype, seed=seed)
    qkv, _ = W.make_values(wl, "cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randn((wl.num_blocks, 2, wl.n_kv_heads, 64, wl.head_dim), generator=g, device="cuda").to(K.F8).view(torch.uint8)
    return wl, qkv, codes, torch.ones((wl.num_blocks, 2, wl.n_kv_heads), device="cuda")


def run(wl, qkv, codes, scales):
    layer = K.layer_for(wl)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    out = torch.full((wl.n_tokens, wl.n_q_heads * wl.head_dim), 7.0, dtype=qkv.dtype, device="cuda")
    layer.attention8(qkv, R.make_kv8_pool(codes, scales), out)
    assert layer.device_error() == 0
    return out


def given(wl, qkv, codes, scales):
    return wl, run(wl, qkv, codes, scales), qkv, codes, scales


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("new", [1, 100], ids=["row", "chunk"])
def test_one_large_value(new, heads, dtype):
    """One element of a block is 2^k times the others' size, and the block's other codes are 0: the other dimensions are made of
    the other blocks.  The block is the first, one in the middle, the last of the history."""
    wl, qkv, codes, scales = batch([(360, new)], heads, dtype)
    ids = K.blocks_of(wl, 0)
    for at in (0, 2, 5):
        for k in (0, 7, 8, 12, 16, 20, 24, 30, 40)[:6 if dtype == "fp16" else 9]:  # (fp16 results end at 2^16)
            c, s = codes.clone(), scales.clone()
            c[ids[at], 1] = 0
            c[ids[at], 1, :, 9, 3] = 0x7e  # 448
            low = -min(k, 14) if dtype == "fp16" else -(k // 2)
            s[:, 1], s[ids[at], 1] = 2.0 ** low, 2.0 ** (low + k)
            B.holds(*given(wl, qkv, c, s))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("seqs", [[(700, 1), (130, 1)], [(300, 150), (0, 70)], [(200, 1), (100, 200), (64, 1)]], ids=["rows", "chunks", "mixed"])
@pytest.mark.parametrize("ends", [9, 20, 48])
def test_scales_far_apart(ends, seqs, heads):
    """Every V tile has a scale of its own from 2^-ends to 2^ends, and every dimension codes in half of the tiles."""
    wl, qkv, codes, scales = batch(seqs, heads, "bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    scales[:, 1] = torch.exp2(torch.randint(-ends, ends + 1, scales[:, 1].shape, generator=g, device="cuda").float())
    codes[:, 1][torch.rand((wl.num_blocks, wl.n_kv_heads, 1, wl.head_dim), generator=g, device="cuda").expand(codes[:, 1].shape) < 0.5] = 0
    B.holds(*given(wl, qkv, codes, scales))


@pytest.mark.parametrize("seqs", [[(500, 1)], [(300, 150)]], ids=["row", "chunk"])
def test_scales_that_are_no_powers_of_two(seqs):
    wl, qkv, codes, scales = batch(seqs, (4, 2, 128), "bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    scales.copy_(torch.exp(torch.randn(scales.shape, generator=g, device="cuda")))
    scales[:, 0] *= 0.25
    scales[:, 1] *= torch.exp(6 * torch.randn(scales[:, 1].shape, generator=g, device="cuda"))
    B.holds(*given(wl, qkv, codes, scales))


@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("seqs", [[(900, 1)], [(800, 100)]], ids=["row", "chunk"])
def test_scales_rise_and_fall(seqs, order):
    """From one block to the next the scale of V goes up (or down) by 2^6, from one end of its range to the other."""
    wl, qkv, codes, scales = batch(seqs, (8, 2, 128), "bf16")
    ids = K.blocks_of(wl, 0)
    e = torch.arange(len(ids), device="cuda").float() * 6 - 45
    scales[ids, 1] = torch.exp2(e if order == "up" else -e)[:, None]
    for b in range(len(ids)):  # a block for each eighth dimension or so
        keep = torch.arange(128, device="cuda") % len(ids) == b
        codes[ids[b], 1, :, :, ~keep] = 0
    B.holds(*given(wl, qkv, codes, scales))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("seqs", [[(200, 1), (63, 1)], [(100, 130), (0, 40)]], ids=["rows", "chunks"])
@pytest.mark.parametrize("k", [-40, -80, -100, 40])
def test_zero_queries_and_key_scales_at_the_ends(k, seqs, heads, dtype):
    """Queries of 0 (every other row of them) average V whatever the keys' scales are; keys that are not seen stay unseen."""
    wl, qkv, codes, scales = batch(seqs, heads, dtype)
    qkv[::2, :heads[0] * heads[2]] = 0
    if k > 0:
        qkv[:, :heads[0] * heads[2]] = 0
    scales[:, 0] = 2.0 ** k
    B.holds(*given(wl, qkv, codes, scales))


def far_apart(wl, scales, heads=None):
    """V scales of every other KV head (or of `heads`) from 2^-12 to 2^12, block by block."""
    g = torch.Generator(device="cuda").manual_seed(9)
    e = torch.randint(-12, 13, scales[:, 1].shape, generator=g, device="cuda").float()
    for h in range(0, wl.n_kv_heads, 2) if heads is None else heads:
        scales[:, 1, h] = torch.exp2(e[:, h])


@pytest.mark.parametrize("heads,seqs", [((64, 8, 128), [(500, 1500), (100, 700)]), ((8, 8, 64), [(0, 3000)]), ((16, 16, 64), [(70, 900), (3, 1)])])
def test_chunks_of_both_kinds_in_one_grid(heads, seqs):
    """Work whose V scales lie far apart between work whose scales do not, many pieces to a CTA: every run has the same bits, and
    they hold."""
    wl, qkv, codes, scales = batch(seqs, heads, "bf16")
    far_apart(wl, scales)
    layer = K.layer_for(wl)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    pool = R.make_kv8_pool(codes, scales)
    outs = torch.zeros((8, wl.n_tokens, heads[0] * heads[2]), dtype=torch.bfloat16, device="cuda")
    for out in outs:
        layer.attention8(qkv, pool, out)
    assert layer.device_error() == 0
    assert all(torch.equal(outs[0], out) for out in outs)
    B.holds(wl, outs[0], qkv, codes, scales)


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_nan_values_with_scales_far_apart(heads, dtype):
    """Slots and blocks of nobody hold NaN; then a NaN value among a chunk's own tokens reaches the rows that see it alone, and
    one of the history all rows."""
    wl, qkv, codes, scales = batch([(100, 300), (10, 20), (130, 1)], heads, dtype)
    hq, hkv, d = heads
    far_apart(wl, scales, range(hkv))
    whole = W.make_custom([(s + n, 1) for s, n in zip(wl.seen, wl.new)], *heads, dtype=dtype)
    whole.block_ids, whole.num_blocks = [np.concatenate([b, np.zeros(1, np.int32)]) for b in wl.block_ids], wl.num_blocks
    codes, scales = K.blanked(whole, codes, scales)
    clean = run(wl, qkv, codes, scales)
    B.holds(wl, clean, qkv, codes, scales)
    clean = clean.view(-1, hq, d)
    ids = K.blocks_of(wl, 0)
    for u, dim in ((50, 1), (100, 0), (127, 63), (128, 5), (255, 17), (399, d - 1)):
        c = codes.clone()
        c[ids[u // 64], 1, hkv - 1, u % 64, dim] = 0x7f + (0x80 if u % 2 else 0)
        got = run(wl, qkv, c, scales).view(-1, hq, d)
        want = torch.zeros_like(got, dtype=torch.bool)
        want[max(u - 100, 0):300, hq - hq // hkv:, dim] = True
        assert torch.equal(torch.isnan(got), want), u
        assert torch.equal(got[~want], clean[~want]), u


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64)])
def test_capacity_call_with_scales_far_apart(heads):
    wl, qkv, codes, scales = batch([(300, 1), (64, 200), (0, 40), (700, 1), (1000, 33)], heads, "bf16")
    far_apart(wl, scales)
    layer = K.layer_for(wl, flags=R.DS_META_CAPACITY, slack=5)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    rows = torch.full((wl.n_tokens + 5, wl.qkv_width), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[:wl.n_tokens] = qkv
    out = torch.full((wl.n_tokens + 5, wl.n_q_heads * wl.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    layer.attention8(rows, R.make_kv8_pool(codes, scales), out)
    assert layer.device_error() == 0 and (out[wl.n_tokens:] == 7).all()
    B.holds(wl, out, qkv, codes, scales)

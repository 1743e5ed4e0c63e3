"""GPU: rotation and append to the 8-bit pool (ds_kv8_rotary_append) against its
definition.

Values are not rotated, so their codes and scales have to be the definition's bit for
bit.  For keys the definition is taken in 64 bits: cosine and sine of the table and
three fp32 rotation steps stay below 2^-21 of |x0| + |x1| of the pair, and an e4m3
rounding is off by at most half a step: 2^-4 of the value, or 2^-10 of a scale below
its normal range.  Scales have to be the definition's unless the tile's largest
magnitude lies that near a power's border.
"""
import numpy as np
import pytest
import torch

import kv8_formula as K
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

F8 = K.F8
MIXED = [(0, 37), (90, 1), (63, 1), (64, 1), (127, 66), (0, 1), (200, 64), (5, 59), (10, 200), (0, 64), (1, 63), (63, 2)]


def same_codes(a, b):
    """Equal as bytes, any NaN equal to any NaN."""
    nan = lambda c: (c & 0x7f) == 0x7f  # noqa: E731
    return ((a == b) | (nan(a) & nan(b))).all()


def check(wl, qkv, before, after, style=R.DS_ROPE_HALF):
    (c0, s0), (c1, s1) = before, after
    _, k, v = K.heads(wl, qkv)
    kr, size = K.rotated(k, K.angles(wl), style)
    want_c, want_s = c0.clone(), s0.clone()  # the V half and what stays exact; the K half is checked on the way
    at = 0
    for i in range(wl.n_seqs):
        seen, n, ids = int(wl.seen[i]), int(wl.new[i]), K.blocks_of(wl, i)
        for b in range(seen // 64, (seen + n - 1) // 64 + 1):
            lo, hi = max(seen - 64 * b, 0), min(seen + n - 64 * b, 64)
            t = slice(at + 64 * b + lo - seen, at + 64 * b + hi - seen)
            new = torch.stack([kr[t], v[t]]).permute(0, 2, 1, 3)  # [2, heads, tokens, d]
            err = torch.stack([size[t] * 2.0 ** -21, torch.zeros_like(size[t])]).permute(0, 2, 1, 3)
            top = torch.nan_to_num(new.abs(), nan=0.0, posinf=float("inf")).amax((2, 3))
            slack = torch.nan_to_num(err, nan=0.0, posinf=0.0).amax((2, 3))
            floor = s0[ids[b]].double() if lo else torch.zeros_like(top)
            least, most = (torch.maximum(K.scale_for((top + e).clamp(min=0)), floor) for e in (-slack, slack))
            s = s1[ids[b]].double()
            assert ((s >= least) & (s <= most)).all(), (i, b, s, least, most)
            assert torch.equal(s[1], least[1])
            want_s[ids[b]] = s.float()
            # earlier codes, rounded anew where the scale grew
            if lo:
                ratio = (s0[ids[b]].double() / s)[..., None, None]
                old = c0[ids[b], :, :, :lo]
                again = (old.view(F8).double() * ratio).float().to(F8).view(torch.uint8)
                want_c[ids[b], :, :, :lo] = torch.where(ratio < 1, again, old)
            # new values exactly, new keys within a rounding
            code = lambda x: (x / s[..., None, None]).clamp(-448, 448).float().to(F8).view(torch.uint8)  # noqa: E731
            want_c[ids[b], :, :, lo:hi] = code(new)
            got = c1[ids[b], 0, :, lo:hi].view(F8).double() * s[0][:, None, None]
            x = new[0].clamp(-448 * s[0][:, None, None], 448 * s[0][:, None, None])
            off = (got - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s[0][:, None, None]) * 1.0001 + err[0]
            assert (off | (torch.isnan(got) & torch.isnan(x))).all(), (i, b)
            want_c[ids[b], 0, :, lo:hi] = c1[ids[b], 0, :, lo:hi]
        at += n
    assert same_codes(c1, want_c), "codes of values, earlier tokens or slots without a token"
    assert torch.equal(s1.nan_to_num(nan=-1.0), want_s.nan_to_num(nan=-1.0))


def run(wl, qkv, codes, scales, style=R.DS_ROPE_HALF, **kw):
    layer = K.layer_for(wl, style, **kw)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    c, s = codes.clone(), scales.clone()
    layer.append8(qkv, R.make_kv8_pool(c, s))
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    return c, s


@pytest.mark.parametrize("style", [R.DS_ROPE_HALF, R.DS_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128), (3, 3, 64), (32, 8, 128), (1, 1, 128), (10, 5, 128)])
def test_matches_definition(heads, dtype, style):
    wl = W.make_custom(MIXED, *heads, dtype=dtype, rope_theta=5.0e5, extra_blocks=3, seed=5)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = K.blanked(wl, *K.made_pool(wl, 1))
    given = qkv.clone()
    check(wl, qkv, (codes, scales), run(wl, qkv, codes, scales, style), style)
    assert torch.equal(qkv, given)


@pytest.mark.parametrize("seqs", [[(0, 1)], [(63, 1)], [(64, 1)], [(4000, 1)], [(0, 300)], [(7, 1)] * 40, [(i, 1) for i in range(130)], [(31, 513), (0, 1)]])
def test_batches(seqs):
    wl = W.make_custom(seqs, 4, 2, 128, dtype="bf16", seed=3)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = K.blanked(wl, *K.made_pool(wl, 1))
    check(wl, qkv, (codes, scales), run(wl, qkv, codes, scales))


def test_random_batches():
    r = np.random.RandomState(11)
    for k in range(12):
        seqs = [(int(r.randint(0, 300)), 1 if r.rand() < 0.5 else int(r.randint(1, 260))) for _ in range(r.randint(1, 30))]
        wl = W.make_custom(seqs, 4, 2, 64, dtype="fp16", seed=k)
        qkv, _ = W.make_values(wl, "cuda")
        codes, scales = K.blanked(wl, *K.made_pool(wl, k))
        check(wl, qkv, (codes, scales), run(wl, qkv, codes, scales))


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-12, 1e-3, 100.0, 1e4, 1e13, 1e17, 1e30])
def test_magnitudes(size):
    """Scales at both ends of their range, zeros, and tiles that have to be rounded anew by many powers."""
    wl = W.make_custom([(70, 1), (0, 1), (64, 30), (100, 40)], 2, 1, 64, dtype="bf16", seed=2)
    qkv, _ = W.make_values(wl, "cuda")
    qkv = (qkv.float() * size).to(torch.bfloat16)
    codes, scales = K.blanked(wl, *K.made_pool(wl, 4))
    check(wl, qkv, (codes, scales), run(wl, qkv, codes, scales))


def test_not_finite():
    wl = W.make_custom([(70, 1), (0, 1), (64, 30), (100, 40)], 2, 1, 64, dtype="bf16", seed=2)
    qkv, _ = W.make_values(wl, "cuda")
    v = qkv.view(wl.n_tokens, 4, 64)[:, 3]
    v[0, 5], v[1, 6], v[5, 7], v[20, 8] = float("nan"), float("inf"), -float("inf"), float("nan")
    v[40] = float("nan")
    codes, scales = K.blanked(wl, *K.made_pool(wl, 4))
    check(wl, qkv, (codes, scales), run(wl, qkv, codes, scales))


def test_growing_block_token_by_token():
    """A block filled by 70 decode steps: each step's scale is what the tokens so far need."""
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.full((2, 2, 2, 64, 64), 0x7f, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, 2, 2), float("nan"), device="cuda")
    for step in range(70):
        wl = W.make_custom([(step, 1)], 2, 2, 64, dtype="fp16", seed=1)
        wl.block_ids, wl.num_blocks = [np.array([1, 0], np.int32)], 2
        qkv = (torch.randn((1, wl.qkv_width), generator=g, device="cuda") * 1.1 ** (step % 60)).half()
        after = run(wl, qkv, codes, scales)
        check(wl, qkv, (codes, scales), after)
        codes, scales = after


def test_second_run_changes_nothing_and_bits_repeat():
    wl = W.make_custom(MIXED, 8, 4, 128, dtype="bf16", seed=6)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = K.made_pool(wl, 1)
    one, two = run(wl, qkv, codes, scales), run(wl, qkv, codes, scales)
    again = run(wl, qkv, *one)
    for other in (two, again):
        assert torch.equal(one[0], other[0]) and torch.equal(one[1], other[1])


def test_capacity_graph_serves_other_batches():
    batches = [W.make_custom(s, 4, 2, 64, dtype="fp16", seed=i) for i, s in enumerate([[(3, 1)] * 5, MIXED, [(0, 400)], [(0, 1)]])]
    blocks = max(w.num_blocks for w in batches)
    for w in batches:
        w.num_blocks = blocks
    big = max(batches, key=lambda w: w.n_tokens)
    st = torch.cuda.Stream()
    layer = R.RaggedLayer(R.params_for(big), 14, 640, 64, 700, stream=st, flags=R.DS_META_CAPACITY)
    rows = torch.zeros((640, big.qkv_width), dtype=torch.float16, device="cuda")
    c, s = (t.clone() for t in K.made_pool(big, 0))
    pool = R.make_kv8_pool(c, s)
    torch.cuda.synchronize()
    layer.build(R.SeqDescs.of(batches[0]), blocks)
    layer.append8(rows, pool)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        layer.build(R.SeqDescs.of(batches[0]), blocks)
        layer.append8(rows, pool)
    for wl in batches + batches[:1]:
        qkv, _ = W.make_values(wl, "cuda")
        codes, scales = K.blanked(wl, *K.made_pool(wl, 9))
        rows.fill_(float("nan"))
        rows[:wl.n_tokens] = qkv
        c.copy_(codes)
        s.copy_(scales)
        torch.cuda.synchronize()
        layer.pack(R.SeqDescs.of(wl), blocks)
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        assert layer.device_error() == 0
        check(wl, qkv, (codes, scales), (c, s))


def test_bad_block_and_position_are_reported():
    """Ids and positions that the metadata's checks did not see (it is replaced on the device) are skipped and reported."""
    wl = W.make_custom([(70, 1), (3, 1)], 2, 2, 64, dtype="fp16", seed=2)
    qkv, _ = W.make_values(wl, "cuda")
    for what, bit in (("block_table", R.DS_DEVERR_BLOCK_ID), ("seq_seen", R.DS_DEVERR_POSITION)):
        layer = K.layer_for(wl)
        layer.build(R.SeqDescs.of(wl), wl.num_blocks)
        torch.cuda.synchronize()
        words = layer.meta_dev.view(torch.int32)
        at = (getattr(layer.meta, what) - layer.meta_dev.data_ptr()) // 4
        words[at + (2 if what == "block_table" else 1)] = wl.num_blocks if what == "block_table" else 72  # the second sequence's
        codes, scales = K.made_pool(wl, 1)
        c, s = codes.clone(), scales.clone()
        layer.append8(qkv, R.make_kv8_pool(c, s))
        assert layer.device_error() == bit
        mine = K.blocks_of(wl, 0)
        rest = torch.ones(wl.num_blocks, dtype=torch.bool, device="cuda")
        rest[mine] = False
        assert torch.equal(c[rest], codes[rest]) and torch.equal(s[rest], scales[rest])
        assert not torch.equal(c[mine], codes[mine])

"""GPU: attention over the 8-bit pool (ds_kv8_blocked_attention) against its formula in
64 bits on the same codes and scales; the tolerance is derived in kv8_formula.attention."""
import numpy as np
import pytest
import torch

import kv8_formula as K
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

MIXED = [(0, 37), (90, 1), (63, 1), (64, 1), (127, 66), (0, 1), (200, 64), (700, 1), (0, 2), (31, 33), (2100, 1), (127, 1), (128, 1)]


def pool_for(wl, seed=1, spread=1.0):
    """A pool in which the batch's tokens are there; slots and blocks of nobody hold NaN codes and scales."""
    codes, scales = K.made_pool(wl, seed, spread)
    whole = W.make_custom([(s + n, 1) for s, n in zip(wl.seen, wl.new)], wl.n_q_heads, wl.n_kv_heads, wl.head_dim, dtype=wl.dtype)
    whole.block_ids, whole.num_blocks = [np.concatenate([b, np.zeros(1, np.int32)]) for b in wl.block_ids], wl.num_blocks
    return K.blanked(whole, codes, scales)


def run(wl, qkv, codes, scales, style=R.DS_ROPE_HALF, rows=1, **kw):
    layer = K.layer_for(wl, style, **kw)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    out = torch.full((wl.n_tokens + rows, wl.n_q_heads * wl.head_dim), 7.0, dtype=qkv.dtype, device="cuda")
    layer.attention8(qkv, R.make_kv8_pool(codes, scales), out)
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    assert (out[wl.n_tokens:] == 7).all()
    return out


@pytest.mark.parametrize("style", [R.DS_ROPE_HALF, R.DS_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128), (3, 3, 64), (16, 4, 128), (1, 1, 128), (8, 1, 64), (8, 2, 64), (4, 2, 128)])
def test_matches_formula(heads, dtype, style):
    wl = W.make_custom(MIXED, *heads, dtype=dtype, rope_theta=5.0e5, extra_blocks=3, seed=5)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    given = (codes.clone(), scales.clone(), qkv.clone())
    out = run(wl, qkv, codes, scales, style)
    K.holds(wl, out, qkv, codes, scales, style)
    assert torch.equal(codes, given[0]) and torch.equal(scales.nan_to_num(), given[1].nan_to_num()) and torch.equal(qkv, given[2])


@pytest.mark.parametrize("heads", [(2, 2, 128), (8, 1, 128), (8, 2, 64)])
@pytest.mark.parametrize("seqs", [[(0, 1)], [(1, 1)], [(62, 1)], [(63, 1)], [(9000, 1)], [(0, 2)], [(0, 700)], [(1000, 300)], [(127, 129)],
                                  [(5, 1)] * 70, [(64 * i, 1) for i in range(40)]])
def test_batches(seqs, heads):
    wl = W.make_custom(seqs, *heads, dtype="bf16", seed=3)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    K.holds(wl, run(wl, qkv, codes, scales), qkv, codes, scales)


@pytest.mark.parametrize("q_size", [1e-20, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("spread", [0.0, 4.0])
@pytest.mark.parametrize("seqs", [[(700, 1), (90, 1)], [(300, 150)]])
def test_magnitudes(seqs, spread, q_size):
    """Queries far from 1 in size (softmax from flat to a single key) and tiles of scales far apart."""
    wl = W.make_custom(seqs, 4, 2, 128, dtype="bf16", seed=3)
    qkv, _ = W.make_values(wl, "cuda")
    qkv[:, :4 * 128] = (qkv[:, :4 * 128].float() * q_size).to(qkv.dtype)
    codes, scales = pool_for(wl, 2, spread)
    K.holds(wl, run(wl, qkv, codes, scales), qkv, codes, scales)


@pytest.mark.parametrize("new", [1, 100])
def test_scales_at_the_ends(new):
    """V tiles of 2^-40 beside tiles of 2^40: what counts is the keys' weights, not the tiles' sizes; and all-zero tiles."""
    wl = W.make_custom([(400, new)], 2, 1, 64, dtype="bf16", seed=3)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    ids = K.blocks_of(wl, 0)
    for size, other in ((2.0 ** -40, 2.0 ** -40), (2.0 ** 40, 2.0 ** 40), (2.0 ** -40, 1.0), (2.0 ** 20, 2.0 ** -20)):
        scales[ids[::2], 1], scales[ids[1::2], 1] = size, other
        K.holds(wl, run(wl, qkv, codes, scales), qkv, codes, scales)
    scales[ids, 1] = 1.0
    codes[ids[1::2]] = 0
    scales[ids[1::2]] = 2.0 ** -40
    K.holds(wl, run(wl, qkv, codes, scales), qkv, codes, scales)


def test_zero_queries_average():
    wl = W.make_custom([(200, 1), (100, 50)], 4, 2, 64, dtype="fp16", seed=3)
    qkv, _ = W.make_values(wl, "cuda")
    qkv[:, :4 * 64] = 0
    codes, scales = pool_for(wl)
    K.holds(wl, run(wl, qkv, codes, scales), qkv, codes, scales)


@pytest.mark.parametrize("seqs", [[(500, 1), (90, 1)], [(200, 60)]])
def test_nan_reaches_its_own_heads_alone(seqs):
    """A NaN key code reaches the rows that see it, of its KV head; a NaN value code its one dimension of them."""
    wl = W.make_custom(seqs, 4, 2, 64, dtype="bf16", seed=3)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    clean = run(wl, qkv, codes, scales)
    ids = K.blocks_of(wl, 0)
    for which, head in ((0, 1), (1, 0)):
        c = codes.clone()
        c[ids[1], which, head, 10, 5] = 0x7f
        got = run(wl, qkv, c, scales)
        rows = int(wl.new[0])
        bad = torch.isnan(got.view(-1, 4, 64))
        want = torch.zeros_like(bad)
        if which == 0:
            want[:rows, 2:4] = True
        else:
            want[:rows, 0:2, 5] = True
        assert torch.equal(bad, want)
        assert torch.equal(got.view(-1, 4, 64)[~bad], clean.view(-1, 4, 64)[~bad])


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
def test_nan_value_of_a_chunks_own_token(heads):
    """The tokens before it do not see it."""
    wl = W.make_custom([(100, 300), (10, 20)], *heads, dtype="bf16", seed=3)
    hq, hkv, d = heads
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    clean = run(wl, qkv, codes, scales).view(-1, hq, d)
    ids = K.blocks_of(wl, 0)
    for u, dim in ((100, 0), (127, 63), (128, 5), (255, 17), (399, d - 1)):
        c = codes.clone()
        c[ids[u // 64], 1, hkv - 1, u % 64, dim] = 0x7f + (0x80 if u % 2 else 0)
        got = run(wl, qkv, c, scales).view(-1, hq, d)
        want = torch.zeros_like(got, dtype=torch.bool)
        want[u - 100:300, hq - hq // hkv:, dim] = True
        assert torch.equal(torch.isnan(got), want)
        # (rows beyond the batch hold what they held; the NaN's own code counts as 0 for the others)
        assert torch.equal(got[~want], clean[~want]), u


@pytest.mark.parametrize("heads,seqs", [((64, 8, 128), [(500, 1500), (100, 700)]), ((8, 8, 64), [(0, 5000)])])
def test_many_tiles_to_a_cta(heads, seqs):
    """Rings and buffers that pass from one tile's work to the next: every run has the same bits, and they hold."""
    wl = W.make_custom(seqs, *heads, dtype="bf16", seed=5)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    layer = K.layer_for(wl)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    pool = R.make_kv8_pool(codes, scales)
    outs = torch.zeros((8, wl.n_tokens, heads[0] * heads[2]), dtype=torch.bfloat16, device="cuda")
    for out in outs:
        layer.attention8(qkv, pool, out)
    assert layer.device_error() == 0
    assert all(torch.equal(outs[0], out) for out in outs)
    K.holds(wl, outs[0], qkv, codes, scales)


def test_bits_repeat_eager_and_captured():
    wl = W.make_custom(MIXED, 8, 2, 128, dtype="bf16", seed=5)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    one = run(wl, qkv, codes, scales)
    assert torch.equal(one, run(wl, qkv, codes, scales))
    st = torch.cuda.Stream()
    layer = K.layer_for(wl, stream=st)
    pool, out = R.make_kv8_pool(codes, scales), torch.zeros_like(one)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        layer.attention8(qkv, pool, out)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:-1], one[:-1])


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64)])
def test_capacity_graph_serves_other_batches(heads):
    lists = [[(300, 1)] * 5, MIXED, [(0, 400)], [(0, 1)], [(1000, 1), (20, 30)]]
    batches = [W.make_custom(s, *heads, dtype="bf16", seed=i) for i, s in enumerate(lists)]
    blocks = max(w.num_blocks for w in batches)
    for w in batches:
        w.num_blocks = blocks
    st = torch.cuda.Stream()
    layer = R.RaggedLayer(R.params_for(batches[0]), 14, 640, 128, 2300, stream=st, flags=R.DS_META_CAPACITY)
    rows = torch.zeros((640, batches[0].qkv_width), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((640, heads[0] * heads[2]), dtype=torch.bfloat16, device="cuda")
    c, s = K.made_pool(batches[0], 0)
    pool = R.make_kv8_pool(c, s)
    torch.cuda.synchronize()
    layer.build(R.SeqDescs.of(batches[0]), blocks)
    layer.attention8(rows, pool, out)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        layer.build(R.SeqDescs.of(batches[0]), blocks)
        layer.attention8(rows, pool, out)
    for wl in batches + batches[:1]:
        qkv, _ = W.make_values(wl, "cuda")
        codes, scales = pool_for(wl, 9)
        rows.fill_(float("nan"))
        rows[:wl.n_tokens] = qkv
        c.copy_(codes)
        s.copy_(scales)
        out.fill_(7)
        torch.cuda.synchronize()
        layer.pack(R.SeqDescs.of(wl), blocks)
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        assert layer.device_error() == 0
        assert (out[wl.n_tokens:] == 7).all()
        K.holds(wl, out, qkv, codes, scales)


@pytest.mark.parametrize("seqs", [[(70, 1), (3, 1)], [(70, 20), (3, 20)]])
def test_bad_block_is_reported(seqs):
    wl = W.make_custom(seqs, 4, 2, 128, dtype="fp16", seed=2)
    qkv, _ = W.make_values(wl, "cuda")
    codes, scales = pool_for(wl)
    layer = K.layer_for(wl)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    torch.cuda.synchronize()
    words = layer.meta_dev.view(torch.int32)
    words[(layer.meta.block_table - layer.meta_dev.data_ptr()) // 4 + 2] = wl.num_blocks  # the second sequence's first block
    out = torch.zeros((wl.n_tokens, 4 * 128), dtype=qkv.dtype, device="cuda")
    layer.attention8(qkv, R.make_kv8_pool(codes, scales), out)
    assert layer.device_error() == R.DS_DEVERR_BLOCK_ID
    want, tol = K.attention(wl, qkv, codes, scales)
    n = int(wl.new[0])  # the first sequence is not touched by it
    assert ((out[:n].double().view(n, 4, 128) - want[:n]).abs() <= tol[:n]).all()


def test_step_after_step_in_one_pool():
    """Prompts in chunks, then decode steps, each appended to the pool and attended over it: every step holds on the
    pool as the appends have left it."""
    g = torch.Generator(device="cuda").manual_seed(5)
    seqs = [(150, 4), (64, 70), (1, 64), (40, 90)]  # (prompt's first chunk, second chunk)
    hq, hkv, d = 8, 2, 128
    total = [a + b + 40 for a, b in seqs]
    plan = W.make_custom([(t - 1, 1) for t in total], hq, hkv, d, dtype="bf16", seed=1)
    codes = torch.full((plan.num_blocks, 2, hkv, 64, d), 0x7f, dtype=torch.uint8, device="cuda")
    scales = torch.full((plan.num_blocks, 2, hkv), float("nan"), device="cuda")
    seen = np.zeros(len(seqs), np.int64)
    for new in [[a for a, _ in seqs], [b for _, b in seqs]] + [[1] * len(seqs)] * 3:
        wl = W.make_custom(list(zip(seen.tolist(), new)), hq, hkv, d, dtype="bf16", seed=1)
        wl.block_ids, wl.num_blocks = plan.block_ids, plan.num_blocks
        qkv = (torch.randn((wl.n_tokens, wl.qkv_width), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
        layer = K.layer_for(wl)
        layer.build(R.SeqDescs.of(wl), wl.num_blocks)
        pool = R.make_kv8_pool(codes, scales)
        out = torch.zeros((wl.n_tokens, hq * d), dtype=torch.bfloat16, device="cuda")
        layer.append8(qkv, pool)
        layer.attention8(qkv, pool, out)
        assert layer.device_error() == 0
        K.holds(wl, out, qkv, codes, scales)
        seen += new


def test_offsets_beyond_32_bits():
    """Blocks whose codes lie more than 4 GiB into the pool: append and attention, decode rows and chunks."""
    import test_gpu_kv8_append as A
    hq, hkv, d, blocks = 16, 8, 128, 33500  # 128 KiB of codes to a block
    wl = W.make_custom([(300, 1), (100, 200), (0, 1)], hq, hkv, d, dtype="bf16", seed=3)
    n = wl.num_blocks
    small_c, small_s = K.made_pool(wl, 2)
    codes = torch.zeros((blocks, 2, hkv, 64, d), dtype=torch.uint8, device="cuda")
    scales = torch.ones((blocks, 2, hkv), device="cuda")
    first = blocks - n
    codes[first:], scales[first:] = small_c, small_s
    assert codes[first:].data_ptr() - codes.data_ptr() > 2 ** 32
    wl.block_ids, wl.num_blocks = [b + first for b in wl.block_ids], blocks
    qkv, _ = W.make_values(W.make_custom([(300, 1), (100, 200), (0, 1)], hq, hkv, d, dtype="bf16", seed=3), "cuda")
    layer = K.layer_for(wl)
    layer.build(R.SeqDescs.of(wl), blocks)
    pool, out = R.make_kv8_pool(codes, scales), torch.zeros((wl.n_tokens, hq * d), dtype=torch.bfloat16, device="cuda")
    layer.append8(qkv, pool)
    layer.attention8(qkv, pool, out)
    assert layer.device_error() == 0
    assert not codes[:first].any() and (scales[:first] == 1).all()
    K.holds(wl, out, qkv, codes, scales)
    wl.block_ids, wl.num_blocks = [b - first for b in wl.block_ids], n
    A.check(wl, qkv, (small_c, small_s), (codes[first:], scales[first:]))

"""GPU: per-head norm + rotary + append (ds_kv_norm_rotary_append) against its
formula in 64 bits.

Tolerance, derived: one rounding to the storage type is half a step, finfo.eps/2
of the value (fp16 subnormals: 2^-25 absolute).  Before it, in fp32: the sum of
squares (16 products and 3 shuffles deep, halved by the root), rsqrtf (2 ulp),
two products, the table's cosine and sine and three rotation steps stay below
2^-19 of |n0| + |n1| of the pair.
"""
import numpy as np
import pytest
import torch

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

MIXED = [(0, 37), (90, 1), (63, 1), (64, 1), (127, 66), (0, 1), (200, 64)]


def formula(wl, qkv, wq, wk, eps, style):
    """(n_q, rotated q, rotated k, v, |n| of the pairs for q and k) in 64 bits."""
    n, hq, hkv, d = wl.n_tokens, wl.n_q_heads, wl.n_kv_heads, wl.head_dim
    x = qkv.double().cpu().numpy().reshape(n, hq + 2 * hkv, d)
    pos = np.concatenate([np.arange(s, s + m) for s, m in zip(wl.seen, wl.new)])
    f = (np.float64(np.float32(wl.rope_theta)) ** (-2.0 * np.arange(d // 2) / d)).astype(np.float32)
    ang = (pos.astype(np.float32)[:, None] * f[None]).astype(np.float64)[:, None, :]
    a, b = (slice(0, d // 2), slice(d // 2, d)) if style == R.DS_ROPE_HALF else (slice(0, d, 2), slice(1, d, 2))

    def one(h, w):
        m = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        m = m * w if w is not None else m
        y, size = np.empty_like(m), np.empty_like(m)
        y[..., a] = m[..., a] * np.cos(ang) - m[..., b] * np.sin(ang)
        y[..., b] = m[..., b] * np.cos(ang) + m[..., a] * np.sin(ang)
        size[..., a] = size[..., b] = np.abs(m[..., a]) + np.abs(m[..., b])
        return m, y, size

    wq, wk = (None if w is None else w.double().cpu().numpy().reshape(-1, d) for w in (wq, wk))
    nq, yq, sq = one(x[:, :hq], wq)
    _, yk, sk = one(x[:, hq:hq + hkv], wk)
    return nq, yq, yk, x[:, hq + hkv:], sq, sk


def close(got, want, size, dtype):
    eps = torch.finfo(W.torch_dtype(dtype)).eps
    got = got.double().cpu().numpy().reshape(want.shape)
    tol = eps / 2 * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -25
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%d of %d off, worst %.3g" % (bad.sum(), bad.size, (np.abs(got - want) - tol).max())


def weights(wl, per_head, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = W.torch_dtype(wl)
    return tuple((1 + 0.3 * torch.randn((h if per_head else 1, wl.head_dim), generator=g, device="cuda")).to(dt)
                 for h in (wl.n_q_heads, wl.n_kv_heads))


def slots(wl):
    """(block, offset) of every packed token."""
    blk, off = [], []
    for s, m, ids in zip(wl.seen, wl.new, wl.block_ids):
        p = np.arange(s, s + m)
        blk.append(np.asarray(ids)[p // 64])
        off.append(p % 64)
    return torch.as_tensor(np.concatenate(blk)).long().cuda(), torch.as_tensor(np.concatenate(off)).long().cuda()


def layer_for(wl, style=R.DS_ROPE_HALF, stream=None, flags=0, slack=0):
    return R.RaggedLayer(R.params_for(wl, style), wl.n_seqs + slack, wl.n_tokens + slack,
                         int(wl.blocks_needed().sum()) + slack, wl.max_len() + slack, stream=stream, flags=flags)


def check_pool(wl, before, after, yk, v, sk):
    blk, off = slots(wl)
    close(after[blk, 0, :, off], yk, sk, wl)
    assert torch.equal(after[blk, 1, :, off].double().cpu(), torch.from_numpy(v))
    rest = after.clone()
    rest[blk, :, :, off] = before[blk, :, :, off]
    assert torch.equal(rest.view(torch.int16), before.view(torch.int16)), "a slot of no new token changed"


@pytest.mark.parametrize("style", [R.DS_ROPE_HALF, R.DS_ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,per_head", [((4, 2, 64), False), ((8, 1, 128), True), ((3, 3, 64), True), ((32, 8, 128), False), ((1, 1, 128), False)])
def test_matches_formula(heads, per_head, dtype, style):
    wl = W.make_custom(MIXED, *heads, dtype=dtype, rope_theta=5.0e5, extra_blocks=3, seed=5)
    qkv, pool = W.make_values(wl, "cuda")
    qkv[5].zero_()  # zero heads: mean 0, so eps alone is under the root
    qkv[7].mul_(1e-3)
    wq, wk = weights(wl, per_head)
    layer = layer_for(wl, style)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    before, given = pool.clone(), qkv.clone()
    width = wl.n_q_heads * wl.head_dim
    qkv_out = torch.full((wl.n_tokens + 1, wl.qkv_width), 7.0, dtype=qkv.dtype, device="cuda")
    q_out = torch.full((wl.n_tokens + 1, width), 7.0, dtype=qkv.dtype, device="cuda")
    eps = 1e-5
    layer.norm_append(R.make_qk_norm(wq, wk, eps, per_head), qkv, pool, qkv_out, q_out)
    torch.cuda.synchronize()
    assert layer.device_error() == 0 and torch.equal(qkv, given)
    nq, yq, yk, v, sq, sk = formula(wl, qkv, wq, wk, np.float32(eps), style)
    close(qkv_out[:-1, :width], nq, np.abs(nq), wl)
    close(q_out[:-1], yq, sq, wl)
    check_pool(wl, before, pool, yk, v, sk)
    assert (qkv_out[:, width:] == 7).all() and (qkv_out[-1] == 7).all() and (q_out[-1] == 7).all()


def test_without_weights_and_in_place():
    wl = W.make_custom(MIXED, 4, 2, 128, dtype="bf16", seed=2)
    qkv, pool = W.make_values(wl, "cuda")
    layer = layer_for(wl)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    before, given = pool.clone(), qkv.clone()
    norm = R.make_qk_norm(None, None, 1e-6)
    other = torch.zeros_like(qkv)
    layer.norm_append(norm, qkv, pool, other)
    second = before.clone()
    layer.norm_append(norm, qkv, second, qkv)
    torch.cuda.synchronize()
    width = wl.n_q_heads * wl.head_dim
    nq, yq, yk, v, sq, sk = formula(wl, given, None, None, np.float32(1e-6), R.DS_ROPE_HALF)
    close(other[:, :width], nq, np.abs(nq), wl)
    assert torch.equal(qkv[:, :width], other[:, :width]) and torch.equal(qkv[:, width:], given[:, width:])
    check_pool(wl, before, pool, yk, v, sk)
    assert torch.equal(second, pool)
    # keys and values alone
    third = before.clone()
    layer.norm_append(norm, given, third)
    torch.cuda.synchronize()
    assert torch.equal(third, pool)


def test_infinities_and_nan_stay_in_their_head():
    wl = W.make_custom([(3, 4), (70, 1)], 4, 2, 64, dtype="fp16", seed=4)
    qkv, pool = W.make_values(wl, "cuda")
    clean = qkv.clone()
    d = wl.head_dim
    qkv[1, d] = float("inf")              # query head 1 of token 1
    qkv[2, 4 * d + 3] = float("nan")      # key head 0 of token 2
    layer = layer_for(wl)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    norm = R.make_qk_norm(None, None)
    a, b = torch.zeros_like(qkv), torch.zeros_like(qkv)
    pa, pb = pool.clone(), pool.clone()
    layer.norm_append(norm, clean, pa, a)
    layer.norm_append(norm, qkv, pb, b)
    torch.cuda.synchronize()
    same = a == b
    same[1, d:2 * d] = True
    assert same.all()
    blk, off = slots(wl)
    same = (pa == pb).clone()
    same[blk[2], 0, 0, off[2]] = True
    assert same.all()


@pytest.mark.parametrize("seen", [0, 8191])
def test_one_token_on_a_stream_of_its_own(seen):
    wl = W.make_custom([(seen, 1)], 64, 8, 128, dtype="bf16", rope_theta=1e6, seed=9)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        qkv, pool = W.make_values(wl, "cuda")
        wq, wk = weights(wl, False)
        layer = layer_for(wl, stream=st)
        layer.build(R.SeqDescs.of(wl), wl.num_blocks)
        before = pool.clone()
        q = torch.zeros((1, 64 * 128), dtype=qkv.dtype, device="cuda")
        layer.norm_append(R.make_qk_norm(wq, wk), qkv, pool, None, q)
        st.synchronize()
        _, yq, yk, v, sq, sk = formula(wl, qkv, wq, wk, np.float32(1e-6), R.DS_ROPE_HALF)
        close(q, yq, sq, wl)
        check_pool(wl, before, pool, yk, v, sk)


def test_captured_call_serves_other_batches():
    """With DS_META_CAPACITY one captured call replays for any batch within the capacities."""
    st = torch.cuda.Stream()
    big = W.make_custom(MIXED, 4, 2, 64, dtype="fp16", seed=1)
    with torch.cuda.stream(st):
        layer = layer_for(big, stream=st, flags=R.DS_META_CAPACITY, slack=8)
        qkv, pool = W.make_values(big, "cuda")
        qkv = torch.cat([qkv, qkv[:8]])
        norm = R.make_qk_norm(*weights(big, False))
        out = torch.full_like(qkv, 7.0)
        layer.build(R.SeqDescs.of(big), big.num_blocks)
        layer.norm_append(norm, qkv, pool, out)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            layer.build(R.SeqDescs.of(big), big.num_blocks)
            layer.norm_append(norm, qkv, pool, out)
        for seqs in ([(0, 1)], [], [(5, 9), (64, 1), (63, 2)], MIXED):
            wl = W.make_custom(seqs, 4, 2, 64, dtype="fp16", seed=6)
            wl.num_blocks = big.num_blocks
            layer.pack(R.SeqDescs.of(wl), big.num_blocks)
            out.fill_(7.0)
            before = pool.clone()
            g.replay()
            st.synchronize()
            assert layer.device_error() == 0
            n = wl.n_tokens
            if n == 0:
                assert torch.equal(pool, before) and (out == 7).all()
                continue
            nq, _, yk, v, _, sk = formula(wl, qkv[:n], *norm.tensors, np.float32(1e-6), R.DS_ROPE_HALF)
            close(out[:n, :256], nq, np.abs(nq), wl)
            check_pool(wl, before, pool, yk, v, sk)
            assert (out[n:] == 7).all()

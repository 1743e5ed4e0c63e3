"""The 8-bit pool's append and attention in 64 bits, for the GPU tests."""
import numpy as np
import torch

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

F8 = torch.float8_e4m3fn


def angles(wl):
    pos = np.concatenate([np.arange(s, s + m) for s, m in zip(wl.seen, wl.new)])
    f = (np.float64(np.float32(wl.rope_theta)) ** (-2.0 * np.arange(wl.head_dim // 2) / wl.head_dim)).astype(np.float32)
    return torch.as_tensor((pos.astype(np.float32)[:, None] * f).astype(np.float64)[:, None], device="cuda")


def rotated(x, ang, style):
    """x [n, heads, d] in 64 bits, rotated; and |x0| + |x1| of each element's pair."""
    d = x.shape[-1]
    a, b = (slice(0, d // 2), slice(d // 2, d)) if style == R.DS_ROPE_HALF else (slice(0, d, 2), slice(1, d, 2))
    y, size = torch.empty_like(x), torch.empty_like(x)
    y[..., a] = x[..., a] * ang.cos() - x[..., b] * ang.sin()
    y[..., b] = x[..., b] * ang.cos() + x[..., a] * ang.sin()
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def heads(wl, qkv):
    """(queries, keys, values) of the packed rows, [n, heads, d] in 64 bits."""
    x = qkv[:wl.n_tokens].double().view(wl.n_tokens, -1, wl.head_dim)
    return x[:, :wl.n_q_heads], x[:, wl.n_q_heads:wl.n_q_heads + wl.n_kv_heads], x[:, wl.n_q_heads + wl.n_kv_heads:]


def scale_for(top):
    """Smallest power of two from 2^-40 to 2^40 with top <= 448 of it (exact: exponents of 64-bit numbers)."""
    m, e = torch.frexp(top.double())
    e = torch.where(torch.isinf(top), 1000, torch.where(m > 0.875, e - 8, e - 9))
    e = torch.where(top > 0, e, -40).clamp(-40, 40)
    return torch.bitwise_left_shift(e.long() + 1023, 52).view(torch.float64)


def made_pool(wl, seed=0, spread=1.0):
    """(codes, scales) of a pool with earlier tokens' codes in every slot: tiles scaled as an append leaves them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (wl.num_blocks, 2, wl.n_kv_heads, 64, wl.head_dim)
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(spread * torch.randn(shape[:3], generator=g, device="cuda"))[..., None, None]
    scales = scale_for(x.abs().amax((3, 4))).float()
    return (x / scales[..., None, None]).to(F8).view(torch.uint8), scales


def blocks_of(wl, i):
    n = (int(wl.seen[i]) + int(wl.new[i]) + 63) // 64
    return torch.as_tensor(np.asarray(wl.block_ids[i])[:n].astype(np.int64), device="cuda")


def blanked(wl, codes, scales):
    """A copy in which everything that no earlier token has is NaN: codes of later slots, blocks not begun and their scales."""
    c, s = torch.full_like(codes, 0x7f), torch.full_like(scales, float("nan"))
    for i in range(wl.n_seqs):
        seen, ids = int(wl.seen[i]), blocks_of(wl, i)
        for b in range((seen + 63) // 64):
            k = min(64, seen - 64 * b)
            c[ids[b], :, :, :k] = codes[ids[b], :, :, :k]
            s[ids[b]] = scales[ids[b]]
    return c, s


def layer_for(wl, style=R.DS_ROPE_HALF, stream=None, flags=0, slack=0):
    return R.RaggedLayer(R.params_for(wl, style), wl.n_seqs + slack, wl.n_tokens + slack,
                         int(wl.blocks_needed().sum()) + slack, wl.max_len() + slack, stream=stream, flags=flags)


def attention(wl, qkv, codes, scales, style=R.DS_ROPE_HALF):
    """(out [n, heads, d] in 64 bits, tolerance).

    Derivation of the tolerance.  Half a step of fp16 is 2^-11 of the value.
      queries: each rotated element is rounded to fp16's 11 bits (below 2^-14 of fp16's range, to 2^-25 of the
        row's largest at most), so a score is off by at most D = 2^-11 sum |q_d k_d| scale; the fp32 sums over d
        and the products with the scales add less than 2^-20 of the same sum.
      weights: w_u changes by a factor within e^(+-D_u), and the normalisation by as much: e^(+-2 max D) in all.
        Each is rounded to fp16 once more (2^-11, in the numerators alone), and exp2's approximation and fp32 sums
        over the keys add 2^-19 and 2^-22 a key at most.
      weights below fp16's normal range, as shares of the largest one or more of its value's tile: 2^-25 of the
        largest element of V a key.
      the result: half a step of the storage type.
    """
    q, _, _ = heads(wl, qkv)
    hq, hkv, d = wl.n_q_heads, wl.n_kv_heads, wl.head_dim
    g = hq // hkv
    scale = d ** -0.5
    dt = W.torch_dtype(wl)
    eps = torch.finfo(dt).eps
    q, size = rotated(q, angles(wl), style)
    out, tol, at = torch.empty_like(q), torch.empty_like(q), 0
    for i in range(wl.n_seqs):
        n, seen, ids = int(wl.new[i]), int(wl.seen[i]), blocks_of(wl, i)
        kv = codes[ids].view(F8).double() * scales[ids].double()[..., None, None]
        k, v = kv.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :seen + n].unbind(0)  # [heads, keys, d]
        for j0 in range(0, n, 128):
            m = min(128, n - j0)
            qq = q[at + j0:at + j0 + m].view(m, hkv, g, d)
            x = torch.einsum("thgd,hud->thgu", qq, k) * scale
            mass = torch.einsum("thgd,hud->thgu", qq.abs() + 2.0 ** -13 * qq.abs().amax(-1, keepdim=True), k.abs()) * scale
            hidden = (torch.arange(seen + n, device="cuda") > seen + j0 + torch.arange(m, device="cuda")[:, None])[:, None, None]
            w = torch.softmax(x.masked_fill(hidden, -np.inf), -1)
            o = torch.einsum("thgu,hud->thgd", w, v)
            size = torch.einsum("thgu,hud->thgd", w, v.abs())
            # a score's own error counts where the key counts; the worst of the row bounds the normalisation
            off = (mass * (2.0 ** -11 + 2.0 ** -20)).masked_fill(hidden, 0)
            worst = off.amax(-1, keepdim=True)
            keys = seen + j0 + m
            t = eps / 2 * o.abs() + size * (torch.expm1(2 * worst) + 2.0 ** -11 + 2.0 ** -19 + keys * 2.0 ** -22) \
                + keys * 2.0 ** -25 * v.abs().amax()
            if dt == torch.float16:
                t = t + 2.0 ** -25
            out[at + j0:at + j0 + m], tol[at + j0:at + j0 + m] = o.reshape(m, hq, d), t.reshape(m, hq, d)
        at += n
    return out, tol


def holds(wl, got, qkv, codes, scales, style=R.DS_ROPE_HALF):
    want, tol = attention(wl, qkv, codes, scales, style)
    got = got[:wl.n_tokens].double().view(want.shape)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%d of %d off, worst %.3g over its tolerance, first at %s" % (
        bad.sum(), bad.numel(), ((got - want).abs() - tol).max(), bad.nonzero()[0].tolist())

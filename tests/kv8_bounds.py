"""The attention over the 8-bit pool in 64 bits, with a bound for every element of its own.

kv8_formula.attention takes the worst score error of a row's keys and the largest value of the pool for every element; here
each key's error counts with the key's weight, and each dimension's with that dimension's values.

Derivation.  fp16's half step is 2^-11 of a value, 2^-22 in two parts, and 2^-25 at least below its normal range.
  scores: a rotated element is off by q = 2^-11 (2^-21 in two parts, for the second part's own half step and the sum of both)
    of itself, or 2^-39 of the row's largest, which is brought to 2^14 or more.  Rotation in fp32, sums over d and the
    products with the scales: less than 2^-20 of the sum of magnitudes.  Together D_u.
  weights: exp2 of an argument y in fp32, y and its parts at most |score| log2(e) + 2 * 48 + 15 in size: the exponent is off by
    2^-23 of that, times ln 2, and exp2 by 2^-21.  Each key's weight is off by E_u = expm1(D_u + that) of itself, above and below
    the fraction.  Above it is rounded once more: r of itself (2^-11 in one part; in two 2^-21, or 2^-17 in chunks whose V scales lie
    far apart, where the parts have 8 bits each), or 2^-25 of the row's largest weight.
  sums: (keys / 16 + 64) 2^-22 of the sums of magnitudes, above and below.
  the result: half a step of the storage type.
"""
import numpy as np
import torch

import kv8_formula as K
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W


def two_parts(wl, new):
    """Whether a sequence's queries and weights go through the products in two parts."""
    return wl.dtype == "fp16" and (new == 1 or wl.head_dim == 64)


def attention(wl, qkv, codes, scales, style=R.DS_ROPE_HALF, weights=2.0 ** -17):
    """(out [n, heads, d] in 64 bits, bound); weights: r of those in two parts."""
    q, _, _ = K.heads(wl, qkv)
    hq, hkv, d = wl.n_q_heads, wl.n_kv_heads, wl.head_dim
    g, scale = hq // hkv, d ** -0.5
    dt = W.torch_dtype(wl)
    eps = torch.finfo(dt).eps
    q, pair = K.rotated(q, K.angles(wl), style)
    out, tol, at = torch.empty_like(q), torch.empty_like(q), 0
    for i in range(wl.n_seqs):
        n, seen, ids = int(wl.new[i]), int(wl.seen[i]), K.blocks_of(wl, i)
        two = two_parts(wl, n)
        kv = codes[ids].view(K.F8).double() * scales[ids].double()[..., None, None]
        k, v = kv.permute(1, 2, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :seen + n].unbind(0)
        keys = seen + n
        for j0 in range(0, n, 64):
            m = min(64, n - j0)
            rows = slice(at + j0, at + j0 + m)
            qq, size = q[rows].view(m, hkv, g, d), pair[rows].view(m, hkv, g, d)
            x = torch.einsum("thgd,hud->thgu", qq, k) * scale
            off = (2.0 ** -21 if two else 2.0 ** -11) * qq.abs() + 2.0 ** -39 * qq.abs().amax(-1, keepdim=True) + 2.0 ** -20 * size
            off = torch.einsum("thgd,hud->thgu", off, k.abs()) * scale
            hidden = (torch.arange(keys, device="cuda") > seen + j0 + torch.arange(m, device="cuda")[:, None])[:, None, None]
            w = torch.softmax(x.masked_fill(hidden, -np.inf), -1)
            reach = x.abs().masked_fill(hidden, 0).amax(-1, keepdim=True) * 1.4427 + 2 * 48 + 15
            e = torch.expm1(off + reach * 2.0 ** -23 * 0.6932 + 2.0 ** -21).masked_fill(hidden, 0)
            sums = (keys / 16 + 64) * 2.0 ** -22
            r = weights if two else 2.0 ** -11
            o = torch.einsum("thgu,hud->thgd", w, v)
            above = torch.einsum("thgu,hud->thgd", w * (e + r + sums) + 2.0 ** -25 * w.amax(-1, keepdim=True) * ~hidden, v.abs())
            below = (w * e).sum(-1, keepdim=True) + sums
            assert below.max() < 0.1, "the bound says nothing for scores as large as these"
            t = (above + o.abs() * below) / (1 - below) * (1 + eps) + eps / 2 * o.abs()
            if dt == torch.float16:
                t = t + 2.0 ** -25
            out[rows], tol[rows] = o.reshape(m, hq, d), t.reshape(m, hq, d)
        at += n
    return out, tol


def holds(wl, got, qkv, codes, scales, style=R.DS_ROPE_HALF, **kw):
    want, tol = attention(wl, qkv, codes, scales, style, **kw)
    got = got[:wl.n_tokens].double().view(want.shape)
    bad = ~((got - want).abs() <= tol)
    first = tuple(bad.nonzero()[0].tolist()) if bad.any() else (0, 0, 0)
    assert not bad.any(), "%d of %d off, the worst by %.3g times its bound, first at %s: %g for %g, bound %g" % (
        bad.sum(), bad.numel(), ((got - want).abs() / tol).nan_to_num(0).max(), first, got[first], want[first], tol[first])

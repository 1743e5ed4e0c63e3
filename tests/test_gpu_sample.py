"""GPU: ds_ragged_sample against its definition in 64 bits.

Tokens are compared for equality: the kernel's weights are within 2^-37 of
exact ones, so a draw differs from the definition's only where u falls that
near a border between two tokens (chance below 1e-5 a row at these sizes).
Log-probabilities: one rounding to 32 bits (2^-24 of the value) and 1e-9.
"""
import math

import numpy as np
import pytest
import torch

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def one_row(x, u, t=1.0, k=0, p=1.0, mp=0.0):
    """(token, log-probability) of a float64 row by the definition."""
    x = np.where(np.isnan(x), -np.inf, x) + 0.0
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if not len(order):
        return -1, -math.inf
    if not t > 0:
        return int(order[0]), 0.0
    m = x[order[0]]
    if k > 0:
        order = order[:k]
    with np.errstate(invalid="ignore"):
        y = np.where(x[order] == m, 0.0, (x[order] - m) / t)
    y = np.where(y * -1.4426950408889634 >= 46, -np.inf, y)
    w = np.exp(y)
    if p < 1:
        w = w[:1 + int(np.searchsorted(np.cumsum(w), max(p, 0.0) * math.fsum(w)))] if p > 0 else w[:1]
    if mp > 0:
        w = w[w >= min(mp, 1.0)]
    by = np.argsort(order[:len(w)])
    c = np.cumsum(w[by])
    u = min(max(u, 0.0), float(np.float32(0.99999994))) if u == u else 0.0
    j = by[min(int(np.searchsorted(c, u * c[-1], side="right")), len(w) - 1)]
    return int(order[j]), float(y[j] - math.log(math.fsum(w)))


def layer_of(rows, stream=None, flags=0, most=0):
    most = max(rows, most, 1)
    layer = R.RaggedLayer(R.make_params(1, 1, 64), most, most, most, 1, stream=stream, flags=flags)
    layer.build(descs(rows), most)
    return layer


def descs(rows):
    return R.SeqDescs([0] * rows, [1] * rows, [np.array([i], np.int32) for i in range(rows)])


def on(v, dt=torch.float32):
    return torch.as_tensor(np.asarray(v), dtype=dt, device="cuda")


def sample(x, u, t=None, k=None, p=None, mp=None, stream=None):
    rows = x.shape[0]
    s = R.make_sampler(on(u), None if t is None else on(t), None if k is None else on(k, torch.int32),
                       None if p is None else on(p), None if mp is None else on(mp))
    tok = torch.full((rows + 2,), 77, dtype=torch.int32, device="cuda")
    lp = torch.full((rows + 2,), 77.0, device="cuda")
    R.ds_ragged_sample(layer_of(rows, stream).meta, x, s, tok, lp, stream)
    torch.cuda.synchronize()
    assert (tok[rows:] == 77).all() and (lp[rows:] == 77).all()
    return tok[:rows].cpu().numpy(), lp[:rows].cpu().numpy()


def check(x, u, t=None, k=None, p=None, mp=None):
    tok, lp = sample(x, u, t, k, p, mp)
    xd = x.double().cpu().numpy()
    f32 = lambda v, i, d: d if v is None else float(np.float32(v[i]))  # noqa: E731
    for i in range(len(tok)):
        want, wlp = one_row(xd[i], f32(u, i, 0), f32(t, i, 1), 0 if k is None else int(k[i]), f32(p, i, 1), f32(mp, i, 0))
        assert tok[i] == want, "row %d: %d, not %d" % (i, tok[i], want)
        assert lp[i] == wlp or abs(lp[i] - wlp) <= 2.0 ** -24 * abs(wlp) + 1e-9, "row %d: %r, not %r" % (i, lp[i], wlp)
    return tok


def logits(rows, vocab, dtype, seed, sigma=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (sigma * torch.randn((rows, vocab), generator=g, device="cuda")).to(DT[dtype])


SETTINGS = {
    "plain": lambda r, n: {},
    "temperature": lambda r, n: dict(t=r.uniform(0.3, 2.0, n)),
    "greedy": lambda r, n: dict(t=np.where(r.rand(n) < 0.5, 0.0, -1.0), k=np.full(n, 3)),
    "top_k": lambda r, n: dict(k=r.randint(1, 300, n), t=r.uniform(0.5, 1.5, n)),
    "top_p": lambda r, n: dict(p=r.uniform(0.05, 0.999, n)),
    "min_p": lambda r, n: dict(mp=r.uniform(0.001, 0.5, n)),
    "all": lambda r, n: dict(t=r.uniform(0.5, 1.5, n), k=r.randint(1, 2000, n), p=r.uniform(0.3, 0.99, n), mp=r.uniform(0, 0.1, n)),
}


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("how", sorted(SETTINGS))
@pytest.mark.parametrize("vocab", [1, 2, 31, 500, 2048, 2049, 5000, 50001])
def test_matches_definition(vocab, how, dtype):
    r = np.random.RandomState(vocab)
    n = 7
    check(logits(n, vocab, dtype, vocab), r.rand(n), **SETTINGS[how](r, n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_largest_vocab(dtype):
    r = np.random.RandomState(1)
    n = 3
    for how in ("temperature", "all"):
        check(logits(n, 262144, dtype, 3), r.rand(n), **SETTINGS[how](r, n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,stride,shift", [(1000, 1003, 1), (999, 999, 3), (4097, 4100, 5), (20000, 20480, 0), (7, 9, 2)])
def test_rows_that_start_anywhere(vocab, stride, shift, dtype):
    r = np.random.RandomState(stride)
    n = 9
    store = torch.full((n * stride + shift + 64,), 60000.0, device="cuda").to(DT[dtype])  # what lies between rows would win
    x = torch.as_strided(store, (n, vocab), (stride, 1), shift)
    x.copy_(logits(n, vocab, dtype, 5))
    check(x, r.rand(n), **SETTINGS["all"](r, n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_equal_logits(dtype):
    n, vocab = 6, 3000
    x = torch.full((n, vocab), -1.5, device="cuda").to(DT[dtype])
    u = [0.0, 0.25, 0.5, 0.75, 0.9999999, 1.0]
    assert list(sample(x, u)[0]) == [0, 750, 1500, 2250, 2999, 2999]
    check(x, u)
    check(x, u, k=[1, 2, 10, 2999, 3000, 5000])
    check(x, u, p=[0.5, 0.25, 0.001, 0.9, 0.0, -1.0])
    check(x, u, k=[100] * n, p=[0.5, 0.1, 0.99, 0.3, 0.02, 0.011])
    check(x, u, mp=[1.0, 2.0, 0.5, 1.0, 0.1, 0.0])
    check(x, u, t=[1e-30, 1e30, float("inf"), 1e-42, 5.0, float("nan")])


def test_ties_at_the_cuts():
    r = np.random.RandomState(0)
    n, vocab = 24, 9000
    x = on(r.randint(-6, 7, (n, vocab)) * 0.5)  # 13 values, hundreds of tokens each
    for dtype in DT:
        check(x.to(DT[dtype]), r.rand(n), k=r.randint(1, 2000, n))
        check(x.to(DT[dtype]), r.rand(n), p=r.uniform(0.01, 0.99, n), t=r.uniform(0.3, 3, n))
        check(x.to(DT[dtype]), r.rand(n), k=r.randint(1, 5000, n), p=r.uniform(0.2, 0.99, n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_masks_infinities_nan_and_zeros(dtype):
    inf, nan = math.inf, math.nan
    n, vocab = 12, 6000
    x = logits(n, vocab, dtype, 8)
    x[0] = -inf                                 # nothing left
    x[1] = nan
    x[2] = -inf
    x[2, 4321] = -60000.0                       # one token left, far down
    x[3, 5], x[3, 17] = inf, inf                # two share the row
    x[4, ::2] = nan
    x[5, :5990] = torch.finfo(x.dtype).min      # masked by the type's lowest value
    x[6] = torch.finfo(x.dtype).min             # a whole row of it
    x[7] = 0.0
    x[7, 1::2] = -0.0                           # equal zeros
    x[8, :] = -inf
    x[8, 100:103] = x[9, 100:103]
    x[10, 0] = torch.finfo(x.dtype).max
    x[11, 3] = -inf
    r = np.random.RandomState(2)
    for how in sorted(SETTINGS):
        check(x, r.rand(n), **SETTINGS[how](r, n))
    check(x, np.where(np.arange(n) % 2, 0.0, 1.0))
    check(x, [nan, -1, 2, inf, -inf, 0.5, 0.3, 0.1, 0.2, 0.99, 0.7, 0.6], k=[-5] * n, p=[nan] * n, mp=[nan] * n)


def test_wide_and_narrow_logits():
    r = np.random.RandomState(4)
    n, vocab = 8, 20000
    for sigma in (1e-4, 0.05, 40.0, 3000.0):
        for dtype in ("fp32", "bf16"):
            for how in ("temperature", "top_k", "top_p", "all"):
                check(logits(n, vocab, dtype, 11, sigma), r.rand(n), **SETTINGS[how](r, n))


def test_every_token_is_reached_in_turn():
    """Flat rows: u at the middle of token i's share picks token i."""
    vocab = 256
    x = torch.zeros((vocab, vocab), device="cuda")
    tok, lp = sample(x, (np.arange(vocab) + 0.5) / vocab)
    assert (tok == np.arange(vocab)).all()
    assert np.abs(lp + math.log(vocab)).max() < 1e-6


def test_no_sequence_and_repeats():
    tok = torch.full((2,), 5, dtype=torch.int32, device="cuda")
    R.ds_ragged_sample(layer_of(0).meta, torch.zeros((1, 8), device="cuda"), R.make_sampler(on([0.1])), tok)
    torch.cuda.synchronize()
    assert (tok == 5).all()
    r = np.random.RandomState(3)
    x, u = logits(40, 70000, "bf16", 1), r.rand(40)
    kw = SETTINGS["top_p"](r, 40)
    a, b = sample(x, u, **kw), sample(x, u, **kw)
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()


def test_two_streams_and_a_captured_call_for_fewer_rows():
    r = np.random.RandomState(6)
    st = [torch.cuda.Stream() for _ in range(2)]
    x = logits(33, 40000, "fp32", 2)
    u, kw = r.rand(33), SETTINGS["all"](r, 33)
    want = check(x, u, **kw)
    for s in st:
        s.wait_stream(torch.cuda.current_stream())
    sp = R.make_sampler(on(u), on(kw["t"]), on(kw["k"], torch.int32), on(kw["p"]), on(kw["mp"]))
    torch.cuda.synchronize()
    out = [torch.zeros(33, dtype=torch.int32, device="cuda") for _ in st]
    layers = [layer_of(33, s) for s in st]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, layer in zip(st, out, layers):
            R.ds_ragged_sample(layer.meta, x, sp, o, None, s)
    torch.cuda.synchronize()
    assert all((o.cpu().numpy() == want).all() for o in out)
    layer = layer_of(33, st[0], R.DS_META_CAPACITY)
    tok = out[0]
    st[0].synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st[0]):
        layer.build(descs(33), 33)
        R.ds_ragged_sample(layer.meta, x, sp, tok, None, st[0])
    for rows in (1, 0, 12, 33):
        layer.pack(descs(rows), 33)
        tok.fill_(-9)
        torch.cuda.synchronize()
        with torch.cuda.stream(st[0]):
            g.replay()
        torch.cuda.synchronize()
        assert (tok[:rows].cpu().numpy() == want[:rows]).all() and (tok[rows:] == -9).all()

"""GPU: rules on logits (ds_ragged_adjust_logits) against their formula in 64 bits.

Tolerance, derived: in fp32 a bias is added, the sum is multiplied by r or by the rounded
1/r, and f c and p are subtracted (f c without a rounding of its own).  Each step is off by half a step (2^-24) of
its result: with X = (|x| + |bias sum|) r', r' the larger of r and 1/r, the sum X, 1/r X, the
product X, the differences X + f c and X + f c + p: at most
2^-24 (5 X + 2 f c + p).  Then one rounding to the storage type.  Elements
that no rule touches, and masks, have to be exact.
"""
import numpy as np
import pytest
import torch

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def meta_for(rows, stream=None, flags=0, capacity=None):
    layer = R.RaggedLayer(R.make_params(1, 1, 64), capacity or rows, capacity or rows, capacity or rows, 1, stream=stream, flags=flags)
    layer.build(descs(rows), capacity or rows)
    return layer


def descs(rows):
    return R.SeqDescs([0] * rows, [1] * rows, [np.array([i], np.int32) for i in range(rows)])


def made(rows, vocab, seed=0, history=60, bias=5, masks=3, unique=True):
    """Rules as host arrays: ids beyond the vocabulary on both sides among them."""
    r = np.random.RandomState(seed)
    d = dict(history=r.randint(-2, vocab + 3, (rows, history)), history_len=r.randint(0, history + 1, rows))
    d["history"][:, ::3] = r.randint(0, max(1, vocab // 9), d["history"][:, ::3].shape)  # common ones
    d["prompt_len"] = r.randint(0, history + 1, rows)
    d["repetition"], d["frequency"], d["presence"] = r.uniform(0.7, 1.5, rows), r.uniform(-0.5, 1, rows), r.uniform(-0.5, 1, rows)
    if bias:
        d["bias_ids"] = np.stack([r.permutation(np.arange(-2, max(vocab, bias) + 2))[:bias] if unique else r.randint(0, min(vocab, 4), bias)
                                  for _ in range(rows)])
        d["bias_ids"][:, 0] = np.clip(d["history"][:, 0], 0, vocab - 1) if unique else d["bias_ids"][:, 0]
        if unique:  # the one above may be there already
            d["bias_ids"][:, 1:][d["bias_ids"][:, 1:] == d["bias_ids"][:, :1]] = -1
        d["bias_values"], d["bias_len"] = r.uniform(-4, 4, (rows, bias)), r.randint(0, bias + 1, rows)
    if masks:
        d["mask"] = r.randint(-2**31, 2**31, (masks, (vocab + 31) // 32 + 2))
        d["mask"][0] = 0
        d["mask"][-1] = -1
        d["mask_row"] = r.randint(-1, masks, rows)
    return {k: v.astype(np.float32 if k in ("repetition", "frequency", "presence", "bias_values") else np.int32) for k, v in d.items()}


def given(d):
    return R.make_logit_rules(**{k: torch.as_tensor(v).cuda().contiguous() for k, v in d.items()})


def formula(x, d):
    """(logits in 64 bits, tolerance before the rounding, tokens touched) of host rows."""
    x = x.astype(np.float64)
    out, tol, touched = x.copy(), np.zeros_like(x), np.zeros(x.shape, bool)
    vocab = x.shape[1]
    for i in range(x.shape[0]):
        rep, freq, pres = (float(d[k][i]) if k in d else n for k, n in (("repetition", 1), ("frequency", 0), ("presence", 0)))
        size = np.abs(x[i])
        if "bias_ids" in d:
            for k in range(d["bias_len"][i] if "bias_len" in d else d["bias_ids"].shape[1]):
                v = d["bias_ids"][i, k]
                if 0 <= v < vocab:
                    out[i, v] += d["bias_values"][i, k]
                    size[v] += abs(d["bias_values"][i, k])
                    touched[i, v] = True
        if "history" in d:
            h = d["history"][i, :min(max(d["history_len"][i], 0), d["history"].shape[1])]
            had = np.unique(h[(h >= 0) & (h < vocab)])
            gen = h[max(d["prompt_len"][i], 0) if "prompt_len" in d else 0:]
            c = np.bincount(gen[(gen >= 0) & (gen < vocab)], minlength=vocab)
            out[i, had] = np.where(out[i, had] > 0, out[i, had] / rep, out[i, had] * rep)
            out[i] -= freq * c + pres * (c > 0)
            r = max(abs(rep), 1 / abs(rep), 1)
            tol[i] = 2.0 ** -24 * (5 * size * r + 2 * abs(freq) * c + abs(pres))
            touched[i, had] = True
        else:
            tol[i] = 2.0 ** -24 * 4 * size
        if "mask" in d:
            m = d["mask_row"][i] if "mask_row" in d else i
            if m >= 0:
                bits = np.unpackbits(d["mask"][m].view(np.uint8), bitorder="little")[:vocab]
                out[i, bits == 0] = -np.inf
    return out, tol, touched


def holds(x, got, d):
    want, tol, touched = formula(x.double().cpu().numpy(), d)
    g = got.double().cpu().numpy()
    gone = np.isneginf(want)
    assert (np.isneginf(g) == gone).all()
    same = ~touched & ~gone
    assert (g[same] == x.double().cpu().numpy()[same]).all()
    eps = torch.finfo(x.dtype).eps
    fine = ~gone
    least = 2.0 ** -25 if x.dtype == torch.float16 else 0  # half a step below fp16's normal range
    bad = np.abs(g[fine] - want[fine]) > (eps / 2 * np.abs(want) + tol * (1 + eps) + least)[fine]
    assert not bad.any(), "%d off" % bad.sum()


def logits(rows, vocab, dtype, seed=0, stride=None, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = stride or vocab
    flat = torch.full((offset + rows * stride,), 9.0, dtype=DT[dtype], device="cuda")
    view = flat[offset:].view(rows, stride)[:, :vocab]
    view.copy_(2.2 * torch.randn((rows, vocab), generator=g, device="cuda"))
    return flat, view


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (5, 33), (2, 2048), (4, 2049), (3, 5001), (1, 32000), (64, 50001), (3, 131072)])
def test_matches_formula(rows, vocab, dtype):
    _, x = logits(rows, vocab, dtype)
    keep = x.clone()
    d = made(rows, vocab, seed=vocab)
    layer = meta_for(rows)
    flat, out = logits(rows, vocab, dtype, 1)
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    assert layer.device_error() == 0
    holds(x, out, d)
    assert torch.equal(x, keep)
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), x)  # in place
    torch.cuda.synchronize()
    assert torch.equal(x, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,xs,xo,ys,yo", [(1000, 1003, 1, 1003, 1), (1000, 1000, 0, 1001, 3), (1000, 1008, 2, 1000, 5), (9, 9, 3, 17, 3), (5000, 5001, 7, 5001, 15)])
def test_rows_at_any_place(dtype, vocab, xs, xo, ys, yo):
    """Rows of another alignment, and nothing between or behind the rows is written."""
    rows = 5
    _, x = logits(rows, vocab, dtype, 0, xs, xo)
    flat, out = logits(rows, vocab, dtype, 1, ys, yo)
    d = made(rows, vocab, seed=4)
    layer = meta_for(rows)  # holds what the metadata points to
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    torch.cuda.synchronize()
    holds(x, out, d)
    rest = torch.ones_like(flat, dtype=torch.bool)
    rest[yo:].view(rows, ys)[:, :vocab] = False
    assert (flat[rest] == 9).all()


@pytest.mark.parametrize("rows,vocab", [(4, 700), (2, 40000)])
@pytest.mark.parametrize("keep", [[], ["history", "history_len"], ["history", "history_len", "repetition"], ["history", "history_len", "prompt_len", "frequency"],
                                  ["history", "history_len", "presence"], ["bias_ids", "bias_values"], ["bias_ids", "bias_values", "bias_len"],
                                  ["mask", "mask_row"], ["mask"], ["history", "history_len", "repetition", "mask", "mask_row"]])
def test_each_rule_alone(keep, rows, vocab):
    d = {k: v for k, v in made(rows, vocab, seed=2, masks=max(3, rows)).items() if k in keep}
    _, x = logits(rows, vocab, "bf16")
    out = torch.zeros_like(x)
    layer = meta_for(rows)  # holds what the metadata points to
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    holds(x, out, d)


def test_biases_of_one_token_add_up_in_order():
    rows, vocab = 3, 5000
    d = made(rows, vocab, seed=1, bias=40, unique=False)
    d["bias_len"][:] = 40
    _, x = logits(rows, vocab, "fp32")
    out = torch.zeros_like(x)
    rules, layer = given(d), meta_for(rows)
    R.ds_ragged_adjust_logits(layer.meta, x, rules, out)
    # 40 biases: 39 sums of magnitudes up to 160, half a step each
    want, tol, _ = formula(x.double().cpu().numpy(), d)
    g = out.double().cpu().numpy()
    fine = ~np.isneginf(want)
    assert (np.abs(g[fine] - want[fine]) <= (tol * 1.01 + 39 * 160 * 1.5 * 2.0 ** -24 + 2.0 ** -24 * np.abs(want))[fine]).all()
    again = torch.zeros_like(x)
    for _ in range(3):
        R.ds_ragged_adjust_logits(layer.meta, x, rules, again)
        assert torch.equal(again, out)


def test_one_token_again_and_again():
    """Counts beyond 16 bits, all of a row's history on one token."""
    rows, vocab, n = 2, 3000, 70000
    d = dict(history=np.full((rows, n), 17, np.int32), history_len=np.array([n, 66000], np.int32), prompt_len=np.array([0, 5], np.int32),
             repetition=np.full(rows, 1.25, np.float32), frequency=np.full(rows, 2.0 ** -10, np.float32), presence=np.full(rows, 0.5, np.float32))
    _, x = logits(rows, vocab, "fp32")
    out = torch.zeros_like(x)
    layer = meta_for(rows)  # holds what the metadata points to
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    holds(x, out, d)


def test_lengths_out_of_range_count_as_the_ends():
    d = made(4, 900, seed=3)
    lens = d["history_len"]
    d["history_len"] = np.array([-5, 0, 10 ** 9, 2 ** 31 - 1], np.int32)
    d["prompt_len"] = np.array([-1, 3, -7, 2 ** 31 - 1], np.int32)
    d["bias_len"] = np.array([-3, 10 ** 6, 2, 2 ** 31 - 1], np.int32)
    _, x = logits(4, 900, "bf16")
    out = torch.zeros_like(x)
    layer = meta_for(4)  # holds what the metadata points to
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    d["bias_len"] = np.array([0, 5, 2, 5], np.int32)
    d["history_len"] = np.array([0, 0, 60, 60], np.int32)
    holds(x, out, d)
    assert lens.shape == (4,)


def test_a_mask_row_that_is_not_there_is_reported():
    d = made(3, 100, seed=3)
    d["mask_row"] = np.array([0, 7, -1], np.int32)
    _, x = logits(3, 100, "bf16")
    out, layer = torch.zeros_like(x), meta_for(3)
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    assert layer.device_error() == R.DS_DEVERR_WORKLIST
    d["mask_row"][1] = -1
    holds(x, out, d)
    assert torch.isneginf(out[0]).all()


def test_infinities_and_nan():
    vocab = 600
    _, x = logits(2, vocab, "fp16")
    x[0, 3], x[0, 4], x[0, 5], x[1, 3] = float("nan"), float("inf"), -float("inf"), 60000.0
    d = dict(history=np.array([[3, 4, 5], [3, 3, 3]], np.int32), history_len=np.array([3, 3], np.int32), prompt_len=np.zeros(2, np.int32),
             repetition=np.array([1.5, 0.5], np.float32), presence=np.array([1.0, 0.0], np.float32))
    out = torch.zeros_like(x)
    layer = meta_for(2)  # holds what the metadata points to
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    assert torch.isnan(out[0, 3]) and out[0, 4] == float("inf") and out[0, 5] == -float("inf")
    assert out[1, 3] == float("inf")  # 120000 is beyond fp16
    rest = torch.ones_like(x, dtype=torch.bool)
    rest[0, 3:6] = rest[1, 3] = False
    assert torch.equal(out[rest], x[rest])


def test_untouched_bits_stay():
    """NaN payloads and negative zeros pass through."""
    x = torch.randint(-2**15, 2**15, (3, 4097), device="cuda", dtype=torch.int16).view(torch.bfloat16)
    d = dict(history=np.zeros((3, 1), np.int32), history_len=np.ones(3, np.int32), repetition=np.full(3, 2.0, np.float32))
    out = torch.zeros_like(x)
    layer = meta_for(3)  # holds what the metadata points to
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
    assert torch.equal(out[:, 1:].view(torch.int16), x[:, 1:].view(torch.int16))


def test_capacity_graph_serves_other_batches_and_leaves_rows_behind():
    cap, vocab = 8, 3001
    st = torch.cuda.Stream()
    layer = meta_for(2, st, R.DS_META_CAPACITY, cap)
    d = made(cap, vocab, seed=6)
    rules = given(d)
    _, x = logits(cap, vocab, "bf16")
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        layer.build(descs(2), cap)
        R.ds_ragged_adjust_logits(layer.meta, x, rules, out, st)
    for rows in (2, 8, 1, 5):
        out.fill_(7)
        torch.cuda.synchronize()
        layer.pack(descs(rows), cap)
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        assert layer.device_error() == 0 and (out[rows:] == 7).all()
        holds(x[:rows], out[:rows], {k: v if k == "mask" else v[:rows] for k, v in d.items()})


def test_draw_from_adjusted_rows():
    """The rules, then the draw, as a server runs them: banned tokens never come, a row without a token gives -1."""
    rows, vocab = 6, 2000
    d = made(rows, vocab, seed=8)
    d["mask_row"] = np.array([1, 0, 1, 1, 2, -1], np.int32)
    _, x = logits(rows, vocab, "bf16")
    layer, out = meta_for(rows), torch.zeros_like(x)
    tokens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    for k in range(10):
        sp = R.make_sampler(torch.full((rows,), k / 10 + 0.05, device="cuda"))
        R.ds_ragged_adjust_logits(layer.meta, x, given(d), out)
        R.ds_ragged_sample(layer.meta, out, sp, tokens)
        got = tokens.cpu().numpy()
        assert got[1] == -1
        w = torch.softmax(out.double(), 1).cpu().numpy()
        for i in (0, 2, 3, 4, 5):
            run = np.cumsum(w[i])
            assert run[got[i]] >= k / 10 + 0.05 - 1e-6 and run[got[i]] - w[i][got[i]] <= k / 10 + 0.05 + 1e-6 and w[i][got[i]] > 0


def test_rows_beyond_32_bits():
    """Rows more than 2^31 elements into a buffer, in place."""
    rows, vocab, stride = 9, 1000, 2 ** 28 + 8
    flat = torch.zeros(rows * stride, dtype=torch.bfloat16, device="cuda")
    x = flat.view(rows, stride)[:, :vocab]
    x.copy_(2.2 * torch.randn((rows, vocab), device="cuda"))
    d, keep, layer = made(rows, vocab, seed=5), x.clone(), meta_for(rows)
    R.ds_ragged_adjust_logits(layer.meta, x, given(d), x)
    torch.cuda.synchronize()
    holds(keep, x, d)
    assert not flat.view(rows, stride)[:, vocab:vocab + 64].any()

"""GPU: rules on logits whose rows of ids and pairs hold what their lengths say and no more: rows of a wider matrix, and a
last row that ends where its memory ends."""
import ctypes

import numpy as np
import pytest
import torch

import test_gpu_adjust_logits as A
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

pytestmark = pytest.mark.gpu


class Memory:
    """Device memory of its own, 4 MiB, so that nothing of another tensor lies behind it."""

    SIZE = 4 << 20

    def __init__(self):
        p = ctypes.c_void_p()
        lib = ctypes.CDLL("libcudart.so.%s" % torch.version.cuda.split(".")[0])
        assert lib.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(self.SIZE)) == 0
        self.lib, self.base = lib, p.value

    def ending_with(self, rows, stride):
        """Address of a matrix of the given 32-bit rows, `stride` apart, the last of which ends the memory."""
        words = (len(rows) - 1) * stride + len(rows[-1])
        at = self.base + self.SIZE - 4 * words
        assert at >= self.base
        for i, r in enumerate(rows):
            r = np.ascontiguousarray(r)
            if r.size:
                assert self.lib.cudaMemcpy(ctypes.c_void_p(at + 4 * i * stride), ctypes.c_void_p(r.ctypes.data), ctypes.c_size_t(r.nbytes), 1) == 0
        return at

    def free(self):
        torch.cuda.synchronize()
        assert self.lib.cudaFree(ctypes.c_void_p(self.base)) == 0


@pytest.mark.parametrize("rows,vocab,history,bias", [(1, 2000, 700, 5), (3, 5001, 60, 40), (4, 40000, 9000, 700), (2, 300, 1, 1)])
def test_the_last_row_ends_the_memory(rows, vocab, history, bias):
    d = A.made(rows, vocab, seed=rows, history=history, bias=bias)
    d["history_len"][-1], d["bias_len"][-1] = history // 3, bias // 3
    _, x = A.logits(rows, vocab, "bf16")
    mems = [Memory() for _ in range(3)]
    rules = A.given(d)
    rules.history = mems[0].ending_with([r[:n] for r, n in zip(d["history"], d["history_len"])], history)
    rules.bias_ids = mems[1].ending_with([r[:n] for r, n in zip(d["bias_ids"], d["bias_len"])], bias)
    rules.bias_values = mems[2].ending_with([r[:n] for r, n in zip(d["bias_values"], d["bias_len"])], bias)
    layer, out = A.meta_for(rows), torch.zeros_like(x)
    R.ds_ragged_adjust_logits(layer.meta, x, rules, out)
    assert layer.device_error() == 0
    A.holds(x, out, d)
    for mem in mems:
        mem.free()


def test_rows_of_a_wider_matrix():
    rows, vocab, n = 3, 5000, 50
    d = A.made(rows, vocab, seed=1, history=n, bias=7)
    wide = {k: torch.zeros((rows, 80), dtype=torch.int32 if k != "bias_values" else torch.float32, device="cuda") for k in ("history", "bias_ids", "bias_values")}
    for k, t in wide.items():
        t[:, 11:11 + d[k].shape[1]] = torch.as_tensor(d[k]).cuda()
    rules = A.given(d)
    rules.history, rules.history_stride = wide["history"].data_ptr() + 44, 80
    rules.bias_ids, rules.bias_values, rules.bias_stride = wide["bias_ids"].data_ptr() + 44, wide["bias_values"].data_ptr() + 44, 80
    _, x = A.logits(rows, vocab, "fp32")
    layer, out = A.meta_for(rows), torch.zeros_like(x)
    R.ds_ragged_adjust_logits(layer.meta, x, rules, out)
    assert layer.device_error() == 0
    A.holds(x, out, d)


@pytest.mark.parametrize("place", ["lines", "single", "biased"])
@pytest.mark.parametrize("size", [1.0, 1e-6, 1e30])
def test_the_quotient_is_off_by_its_rounding(place, size):
    """z / r and z * r are off by half a step of fp32 and 2^-45 of themselves at most, wherever the token lies."""
    rows, vocab = 64, 4000
    r = np.random.RandomState(3)
    flat, x = A.logits(rows, vocab, "fp32")
    x *= size
    d = dict(history=np.tile(np.arange(vocab, dtype=np.int32), (rows, 1)), history_len=np.full(rows, vocab, np.int32),
             repetition=np.concatenate([[1.3, 0.7, 1.9999999, 2.0 ** 60], r.uniform(0.5, 2, rows - 4)]).astype(np.float32),
             prompt_len=np.full(rows, vocab, np.int32))
    if size > 1:
        d["repetition"][3] = 1.1
    if place == "biased":
        d["bias_ids"] = np.stack([r.permutation(vocab)[:2000] for _ in range(rows)]).astype(np.int32)
        d["bias_values"] = np.zeros((rows, 2000), np.float32)
    out = torch.zeros(rows * vocab + 1, device="cuda")[1 if place == "single" else 0:][:rows * vocab].view(rows, vocab)
    layer = A.meta_for(rows)
    R.ds_ragged_adjust_logits(layer.meta, x, A.given(d), out)
    assert layer.device_error() == 0
    z, rep, got = x.double().cpu().numpy(), d["repetition"].astype(np.float64)[:, None], out.double().cpu().numpy()
    want = np.where(z > 0, z / rep, z * rep)
    # half a step is 2^-24 of the power of two at or below the number
    m, e = np.frexp(np.abs(want))
    assert (np.abs(got - want) <= np.ldexp(1.0, e - 25) + 2.0 ** -45 * np.abs(want) + 2.0 ** -150).all()


def test_repetitions_at_the_ends():
    """r of 0, infinite, subnormal and negative, and infinite logits: what fp32 gives for z / r and z * r."""
    reps = np.array([0.0, np.inf, 2.0 ** -140, -2.0, 2.0 ** 120, 1e-39, 1.7], np.float32)
    rows, vocab = len(reps), 64
    _, x = A.logits(rows, vocab, "fp32")
    x[:, 0], x[:, 1], x[:, 2], x[:, 3], x[:, 4] = np.inf, -np.inf, np.nan, 0.0, 3e38
    d = dict(history=np.tile(np.arange(vocab, dtype=np.int32), (rows, 1)), history_len=np.full(rows, vocab, np.int32), repetition=reps,
             prompt_len=np.full(rows, vocab, np.int32))
    out = torch.zeros_like(x)
    layer = A.meta_for(rows)
    R.ds_ragged_adjust_logits(layer.meta, x, A.given(d), out)
    assert layer.device_error() == 0
    with np.errstate(all="ignore"):
        z = x.cpu().numpy()
        want = np.where(z > 0, z / reps[:, None], z * reps[:, None])
    got = out.cpu().numpy()
    # 1 / r is infinite for subnormal r, where z / r may not be: left out
    keep = ~((np.abs(reps) > 0) & (np.abs(reps) < 2.0 ** -126))[:, None] | (z <= 0) | ~np.isfinite(want)
    assert (np.isnan(got) == np.isnan(want))[keep].all()
    both = keep & ~np.isnan(want)
    assert np.allclose(got[both], want[both], rtol=2.0 ** -22, atol=0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("repeated", [False, True])
@pytest.mark.parametrize("rows,vocab,shift", [(3, 5000, 0), (2, 3001, 1), (2, 40000, 0)])
def test_the_longest_bias_lists(rows, vocab, shift, repeated, dtype):
    """2046 pairs: more than a CTA's threads, tokens that come again far down the list, under masks, out of place and in place."""
    n = 2046
    r = np.random.RandomState(vocab)
    d = A.made(rows, vocab, seed=5, history=200, bias=0, masks=3)
    d["mask_row"] = np.arange(rows, dtype=np.int32) % 3
    ids = np.stack([r.permutation(vocab)[:n] for _ in range(rows)])
    if repeated:  # entry j + 1000 is entry j's token once more, and again at the end
        ids[:, 1000:1500] = ids[:, 0:500]
        ids[:, n - 40:] = ids[:, 490:530]
    d["bias_ids"], d["bias_values"] = ids.astype(np.int32), r.uniform(-4, 4, (rows, n)).astype(np.float32)
    d["bias_len"] = np.array([n, n, 600][:rows], np.int32)
    flat = torch.zeros(rows * vocab + 8, dtype=A.DT[dtype], device="cuda")
    _, given = A.logits(rows, vocab, dtype)
    x = flat[shift:shift + rows * vocab].view(rows, vocab)
    x.copy_(given)
    layer, out, rules = A.meta_for(rows), torch.zeros_like(given), A.given(d)
    R.ds_ragged_adjust_logits(layer.meta, x, rules, out)
    assert layer.device_error() == 0 and torch.equal(x, given)
    A.holds(given, out, d)  # (three entries of a token: two sums of magnitudes below 12, within the bound's 5 half steps of X)
    R.ds_ragged_adjust_logits(layer.meta, x, rules, x)
    torch.cuda.synchronize()
    assert torch.equal(x, out)

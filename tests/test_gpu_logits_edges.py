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

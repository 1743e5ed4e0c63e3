"""Subprocess half of test_gpu_kv8_runout.py: drives a test build of the library
(compiled with -DDSR_TEST_WAIT_RUNOUT: every mbarrier wait bounded at ~1 ms, and a device
word that withholds copies from the 8-bit pool).

    python kv8_runout_probe.py <path of the test build's libds_ragged.so>

For several points from which on a decode warp or a prefill CTA gets no more codes: the
waits behind it run out with nothing in flight, the call comes back promptly with
DS_DEVERR_WORKLIST in the batch's error word, and the next call is right.
Prints one JSON line; exit status 0 when all hold.
"""
import ctypes
import json
import os
import sys
import time

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import torch  # noqa: E402

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R  # noqa: E402
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W  # noqa: E402


def runs(lib):
    import kv8_formula as K
    lib.ds_test_withhold_kv8.restype = ctypes.c_int32
    lib.ds_test_withhold_kv8.argtypes = [ctypes.c_int32]
    res = []
    for heads, seqs, points in (((8, 1, 128), [(2000, 1), (300, 1), (64 * 33, 1)], (1, 2)), ((4, 4, 64), [(700, 1)] * 3, (1, 2)),
                                ((8, 1, 128), [(300, 40)], (1, 2, 3, 4, 5, 7, 8, 9)), ((4, 2, 64), [(90, 500), (0, 33)], (1, 3, 6))):
        wl = W.make_custom(seqs, *heads, dtype="bf16", seed=3)
        qkv, _ = W.make_values(wl, "cuda")
        codes, scales = K.made_pool(wl)
        pool, out = R.make_kv8_pool(codes, scales), torch.zeros((wl.n_tokens, heads[0] * heads[2]), dtype=torch.bfloat16, device="cuda")
        want, tol = K.attention(wl, qkv, codes, scales)
        layer = K.layer_for(wl)
        for n in points:
            layer.build(R.SeqDescs.of(wl), wl.num_blocks)
            torch.cuda.synchronize()
            assert lib.ds_test_withhold_kv8(n) == R.DS_OK
            t0 = time.perf_counter()
            layer.attention8(qkv, pool, out)
            torch.cuda.synchronize()
            took, err = time.perf_counter() - t0, layer.device_error()
            assert lib.ds_test_withhold_kv8(0) == R.DS_OK
            layer.build(R.SeqDescs.of(wl), wl.num_blocks)  # a fresh upload clears the error word
            out.fill_(7.0)
            layer.attention8(qkv, pool, out)
            torch.cuda.synchronize()
            right = ((out.double().view(want.shape) - want).abs() <= tol).all()
            res.append(dict(heads=heads, n=n, took_s=took, error=err, after=layer.device_error(), right=bool(right)))
    return all(r["error"] == R.DS_DEVERR_WORKLIST and r["took_s"] < 10 and r["after"] == 0 and r["right"] for r in res), res


def main(lib_path):
    R.LIB_PATH = lib_path
    ok, res = runs(R.load())
    print(json.dumps(dict(ok=ok, runs=res)), flush=True)
    return 0 if ok else 1


if __name__ == "__main__":
    sys.exit(main(sys.argv[1]))

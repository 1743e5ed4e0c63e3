"""Subprocess half of test_gpu_operators_runout.py: drives a test build of the
library (compiled with -DDSR_TEST_WAIT_RUNOUT: every mbarrier wait bounded at
~1 ms, and a device word that withholds fetches of the large low-rank tiles).

    python operators_runout_probe.py <path of the test build's libds_ragged.so>

For several points of a tile from which on nothing is fetched: the waits behind it
run out with nothing in flight, the call comes back promptly with
DS_DEVERR_WORKLIST in the plan's error word, rows of other sequences and of
small tiles are untouched by it, and the next call is right.
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


def withheld_copies(lib):
    import test_gpu_lora as L
    lib.ds_test_withhold_lora.restype = ctypes.c_int32
    lib.ds_test_withhold_lora.argtypes = [ctypes.c_int32]
    res = []
    # one tile: a cluster of 8 with 8 fetches each for the first product, 4 for the second
    # 12 tiles: clusters of 8; 160: of 1, with 4 and 5
    for new, rank, wi, wo, dtype, points in (
            ([100, 3], 64, 4096, 2048, "bf16", (1, 2, 4, 5, 8, 9, 10, 11, 12)),
            ([100, 3], 128, 4096, 2048, "fp16", (1, 3, 5, 8, 9, 10, 11, 12)),
            ([70] * 12, 16, 1000, 1496, "fp16", (1, 2, 3, 4)),
            ([128] * 159 + [40], 40, 256, 320, "bf16", (1, 3, 5, 6, 7, 8, 9))):
        d = L.make(new, list(range(len(new))), len(new), rank, wi, wo, dtype, seed=rank)
        want, tol = L.formula(d)
        lora = R.make_lora(d["a"], d["b"], d["scale"])
        plan = R.LoraPlan(len(new), sum(new))
        out = torch.empty_like(d["base"])
        for n in points:
            plan.build(d["new"], d["which"], d["na"])
            out.fill_(7.0)
            torch.cuda.synchronize()
            assert lib.ds_test_withhold_lora(n) == R.DS_OK
            t0 = time.perf_counter()
            R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out)
            torch.cuda.synchronize()
            took = time.perf_counter() - t0
            err = plan.device_error()
            assert lib.ds_test_withhold_lora(0) == R.DS_OK
            small = ((out[100:].double() - want[100:]).abs() <= tol[100:]).all() if new[-1] == 3 else True
            plan.build(d["new"], d["which"], d["na"])  # a fresh upload clears the error word
            out.fill_(7.0)
            R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out)
            torch.cuda.synchronize()
            after = plan.device_error()
            right = ((out.double() - want).abs() <= tol).all()
            res.append(dict(tokens=len(out), rank=rank, n=n, took_s=took, error=err, small=bool(small), after=after,
                            right=bool(right)))
    ok = all(r["error"] == R.DS_DEVERR_WORKLIST and r["took_s"] < 10 and r["small"] and r["after"] == 0 and r["right"] for r in res)
    return ok, res


def main(lib_path):
    R.LIB_PATH = lib_path
    ok, res = withheld_copies(R.load())
    print(json.dumps(dict(ok=ok, runs=res)), flush=True)
    return 0 if ok else 1


if __name__ == "__main__":
    sys.exit(main(sys.argv[1]))

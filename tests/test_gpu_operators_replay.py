"""GPU: replays of captured operator calls whose plan or batch has changed since."""
import numpy as np
import pytest
import torch

import test_gpu_lora as L
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,rank", [("bf16", 16), ("fp16", 64), ("bf16", 128)])
def test_replay_with_more_adapters_than_were_captured(dtype, rank):
    """Tokens of adapters that the captured weights lack keep their rows, and the error word says so."""
    st = torch.cuda.Stream()
    new, known = [1, 40, 3, 130, 1, 33], [0, 1, 2, 0, -1, 2]
    d = L.make(new, known, 3, rank, 512, 320, dtype, seed=2)
    lora = R.make_lora(d["a"], d["b"], d["scale"])
    plan = R.LoraPlan(8, sum(new), flags=R.DS_META_CAPACITY, stream=st)
    out = torch.full_like(d["base"], 7.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        plan.build(new, known, 3)
        R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out, st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        plan.build(new, known, 3)
        R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out, st)
    want, tol = L.formula(d)
    for which, n_adapters in (([0, 3, 2, 4, 1000, 2], 1001), (known, 3), ([2 ** 31 - 2] * 6, 2 ** 31 - 1)):
        plan.pack(new, which, n_adapters)
        out.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        st.synchronize()
        beyond = torch.as_tensor(np.repeat(np.array(which) >= 3, new), device="cuda")
        assert (plan.device_error() == R.DS_DEVERR_WORKLIST) == bool(beyond.any())
        assert (out[beyond] == 7).all()
        there = ~beyond & torch.as_tensor(np.repeat(np.array(which) == known, new), device="cuda")
        assert ((out[there].double() - want[there]).abs() <= tol[there]).all()
    plan.pack(new, known + [], 4)  # packed for another number: refused where the call is made
    with pytest.raises(R.DSError):
        R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out, st)

"""GPU: infinite elements through ds_ragged_lora, where the kernels pad the rank."""
import pytest
import torch

import test_gpu_lora as L

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 56, 64, 72, 104, 128])
@pytest.mark.parametrize("new", [[3, 1], [100, 40]], ids=["small_tiles", "large_tiles"])
def test_an_infinite_input_gives_the_formulas_infinities(new, rank, dtype):
    """Positive adapters: out is +inf wherever x has a +inf, -inf for a -inf, and NaN for nothing."""
    d = L.make(new, [0, 1], 2, rank, 200, 136, dtype, seed=rank)
    d["a"], d["b"] = d["a"].abs() + 0.01, d["b"].abs() + 0.01
    clean = L.check(d)
    d["x"][0, 5], d["x"][2, 199], d["x"][-1, 0] = INF, -INF, INF
    out = L.run(d)
    assert (out[0] == INF).all() and (out[2] == -INF).all() and (out[-1] == INF).all()
    assert torch.equal(out[3:-1], clean[3:-1]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("rank", [16, 64, 72])
@pytest.mark.parametrize("new", [[3, 1], [100, 40]], ids=["small_tiles", "large_tiles"])
def test_an_infinite_weight_leaves_large_neighbours_finite(new, rank):
    """fp16: v beyond the type's range beside an infinite one is scaled down, not another infinity."""
    d = L.make(new, [0, 1], 2, rank, 256, 136, "fp16", seed=rank, size=1e4)
    d["x"], d["a"] = d["x"].abs() + 1, d["a"].abs() + 1
    assert (d["x"].double() @ d["a"][0].double().T).min() > 1e6
    d["a"][:, 3, 7] = INF
    d["b"][:, :, 3] = 1
    d["b"][:, :, 5] = -1e-3  # v5 is finite: +inf - finite
    out = L.run(d)
    assert (out == INF).all()

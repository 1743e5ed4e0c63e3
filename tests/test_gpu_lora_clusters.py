"""GPU: ds_ragged_lora at numbers of tiles on both sides of each cluster size's limit."""
import pytest

import test_gpu_lora as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [32, 72, 128])
@pytest.mark.parametrize("tiles", [15, 16, 36, 37, 74, 75, 77, 153])
def test_large_tiles(tiles, rank):
    new = [128] * (tiles - 1) + [33]
    L.check(L.make(new, [i % 5 for i in range(tiles)], 5, rank, 520, 328, "fp16" if tiles % 2 else "bf16", seed=tiles))


@pytest.mark.parametrize("rank", [32, 72, 128])
@pytest.mark.parametrize("tiles", [15, 16, 36, 37, 74, 75, 77, 153, 305])
def test_small_tiles(tiles, rank):
    L.check(L.make([1] * tiles, list(range(tiles)), tiles, rank, 520, 328, "bf16" if tiles % 2 else "fp16", seed=tiles))


@pytest.mark.parametrize("rank", [32, 128])
@pytest.mark.parametrize("small,large", [(3, 1), (20, 3), (40, 6), (90, 12), (8, 30), (200, 20)])
def test_both_kinds_side_by_side(small, large, rank):
    new, which = [1] * small + [128] * large, list(range(small)) + list(range(large))
    L.check(L.make(new, which, small + large, rank, 520, 328, "bf16", seed=small))

"""GPU: rows that leave ds_ragged_sample by every way out, side by side in one launch
and in clusters of every size, against the definition in 64 bits."""
import numpy as np
import pytest

import test_gpu_sample as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(5, 3000), (18, 17000), (36, 17000), (72, 17000), (150, 17000), (300, 700)])
def test_every_way_out_side_by_side(rows, vocab, dtype):
    """First of the largest, nothing left, few gathered tokens, cuts ranked among many, and the plain running weight."""
    r = np.random.RandomState(rows)
    x = S.logits(rows, vocab, dtype, rows, sigma=2.0)
    x[::7] = float("-inf")
    x[3::7] = 1.0
    x[4::7, ::3] = float("nan")
    t = np.where(np.arange(rows) % 5 == 1, 0.0, r.uniform(0.4, 2.0, rows))
    k = np.where(np.arange(rows) % 3 == 0, r.randint(1, 600, rows), 0)
    p = np.where(np.arange(rows) % 4 == 0, r.uniform(0.2, 0.99, rows), 1.0)
    mp = np.where(np.arange(rows) % 6 == 5, 0.05, 0.0)
    u = r.rand(rows)
    first = S.check(x, u, t=t, k=k, p=p, mp=mp)
    for _ in range(20):
        assert (S.sample(x, u, t=t, k=k, p=p, mp=mp)[0] == first).all()

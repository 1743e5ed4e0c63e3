"""GPU: ds_kv_norm_rotary_append with qkv_out = qkv, against the same call with rows of their own."""
import pytest
import torch

import test_gpu_norm_append as A
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("style", [R.DS_ROPE_HALF, R.DS_ROPE_INTERLEAVED])
@pytest.mark.parametrize("heads,dtype", [((64, 8, 128), "bf16"), ((32, 32, 128), "fp16"), ((4, 2, 64), "bf16"), ((8, 1, 64), "fp16")])
def test_in_place_gives_the_same_bits(heads, dtype, style):
    wl = W.make_custom(A.MIXED + [(5, 700), (300, 1), (0, 256)], *heads, dtype=dtype, seed=8)
    qkv, pool = W.make_values(wl, "cuda")
    layer = A.layer_for(wl, style)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    norm = R.make_qk_norm(*A.weights(wl, True), 1e-5, per_head=True)
    width = wl.n_q_heads * wl.head_dim
    rows, turned = torch.empty_like(qkv), torch.empty((wl.n_tokens, width), dtype=qkv.dtype, device="cuda")
    first = pool.clone()
    layer.norm_append(norm, qkv, first, rows, turned)
    for _ in range(5):
        mine, again, second = qkv.clone(), torch.empty_like(turned), pool.clone()
        layer.norm_append(norm, mine, second, mine, again)
        torch.cuda.synchronize()
        assert torch.equal(mine[:, :width], rows[:, :width]) and torch.equal(mine[:, width:], qkv[:, width:])
        assert torch.equal(again, turned) and torch.equal(second, first)

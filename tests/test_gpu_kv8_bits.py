"""GPU: the bits that queries and softmax weights keep in attention over the 8-bit pool (kv8_bounds derives the bound): 22 in
fp16 layers' rows and their chunks of d = 64, 11 else; and a key far ahead of the others gives its value."""
import pytest
import torch

import kv8_bounds as B
import kv8_formula as K
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from test_gpu_kv8_scales import batch, given, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [1.0, 4.0])
@pytest.mark.parametrize("seqs", [[(90, 1), (63, 1), (130, 1), (5, 1)], [(30, 90), (0, 64), (60, 2)]], ids=["rows", "chunks"])
@pytest.mark.parametrize("heads,dtype", [((4, 2, 64), "fp16"), ((8, 1, 64), "fp16"), ((8, 2, 128), "fp16"), ((3, 3, 128), "fp16"),
                                         ((4, 2, 64), "bf16"), ((8, 2, 128), "bf16")])
def test_bits_of_queries_and_weights(heads, dtype, seqs, size):
    """Scores up to about 6 and 24 of values that cancel: many results are small beside the sum of their terms, so that their own
    rounding does not hide the terms'."""
    wl, qkv, codes, scales = batch(seqs, heads, dtype)
    qkv[:, :heads[0] * heads[2]] *= size if B.two_parts(wl, int(wl.new[0])) else size / 2
    scales[:, 1] = 2.0 ** 6  # the results' subnormals stay out of it
    B.holds(*given(wl, qkv, codes, scales), weights=2.0 ** -21)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("new", [1, 150], ids=["row", "chunk"])
@pytest.mark.parametrize("key_scale", [2.0 ** -4, 1.0, 2.0 ** 4, 2.0 ** 8])
@pytest.mark.parametrize("winner", [0, 77, 299])
def test_a_key_far_ahead(winner, key_scale, new, heads, dtype):
    """Scores times log2(e) up to 2^23.6; one key is ahead of the others by 2^10 or more, so every other weight is 0."""
    wl, qkv, codes, scales = batch([(300, new)], heads, dtype)
    hq, hkv, d = heads
    # queries and keys in the last dimension alone: its pair turns by less than 0.1 at these positions
    qkv[:, :hq * d] = 0
    qkv[:, :hq * d].view(wl.n_tokens, hq, d)[:, :, d - 1] = 600.0
    ids = K.blocks_of(wl, 0)
    codes[:, 0] = 0
    codes[:, 0, :, :, d - 1] = 0x50  # 8
    codes[ids[winner // 64], 0, :, winner % 64, d - 1] = 0x7e  # 448
    scales[:, 0] = key_scale
    g = torch.Generator(device="cuda").manual_seed(winner)
    e = torch.randint(-6, 7, (wl.num_blocks, hkv), generator=g, device="cuda").float()
    scales[:, 1] = torch.exp2(e)
    out = run(wl, qkv, codes, scales).double().view(-1, hkv, hq // hkv, d)
    v = codes[ids[winner // 64], 1, :, winner % 64].view(K.F8).double() * scales[ids[winner // 64], 1].double()[:, None]
    r = 2.0 ** -17 if B.two_parts(wl, new) else 2.0 ** -11
    bound = v.abs() * (torch.finfo(qkv.dtype).eps / 2 * (1 + r) + r + 2.0 ** -18) + 2.0 ** -25
    assert ((out - v[None, :, None]).abs() <= bound[None, :, None]).all()

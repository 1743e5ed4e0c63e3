"""GPU: what follows an attention call on its stream finds all of `out`, the chunks' rows too, where the decode rows' kernel runs
beside the chunks' and is the call's last launch (no row is split, so there is no merge): a copy in stream order, a
kernel launched as a programmatic dependent (pdl_follower.cu), eager and captured."""
import ctypes
import os
import subprocess

import pytest
import torch

from ragged_blocked_kv_raggedbatch_gb300 import build as B
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def follow(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("follower") / "libfollower.so")
    r = subprocess.run([B._nvcc()] + B.ARCH + ["-std=c++17", "-shared", "-Xcompiler", "-fPIC", os.path.join(HERE, "pdl_follower.cu"), "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    fn = ctypes.CDLL(lib).follow
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]

    def call(src, dst, stream):
        assert fn(src.data_ptr(), dst.data_ptr(), src.numel() * src.element_size() // 16, stream.cuda_stream) == 0
    return call


CALLS = ["attention8", "attention", "fused"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("heads", [(16, 2, 128), (4, 4, 64)], ids=["gqa", "mha"])
@pytest.mark.parametrize("flags", [0, R.DS_META_CAPACITY], ids=["batch", "capacity"])
def test_follower_finds_every_row(follow, call, heads, flags):
    # rows of one block beside chunks that take hundreds of times as long
    wl = W.make_custom([(20, 1), (4000, 1500), (40, 1), (5, 1), (3000, 700)], *heads, dtype="bf16", seed=3)
    hq, hkv, d = heads
    qkv, pool16 = W.make_values(wl, "cuda")
    codes = pool16.to(torch.float8_e4m3fn).view(torch.uint8)
    pool8 = R.make_kv8_pool(codes, torch.ones(codes.shape[:3], device="cuda"))
    st = torch.cuda.Stream()
    layer = R.RaggedLayer(R.params_for(wl), wl.n_seqs, wl.n_tokens, int(wl.blocks_needed().sum()), wl.max_len(), stream=st, flags=flags)
    layer.build(R.SeqDescs.of(wl), wl.num_blocks)
    if not flags:
        assert layer.meta.n_decode_items == layer.meta.n_decode_seqs == 3 and layer.meta.n_prefill_tiles > 0
    out = torch.zeros((wl.n_tokens, hq * d), dtype=torch.bfloat16, device="cuda")
    seen, seen_late = torch.zeros_like(out), torch.zeros_like(out)
    torch.cuda.synchronize()

    def step():
        out.fill_(7.0)
        if call == "attention8":
            layer.attention8(qkv, pool8, out)
        elif call == "attention":
            layer.attention(qkv, pool16, out)
        else:
            layer.fused(qkv, pool16, out)
        follow(out, seen, st)
        seen_late.copy_(out)

    with torch.cuda.stream(st):
        step()
    st.synchronize()
    assert layer.device_error() == 0
    want = out.clone()
    assert not (want == 7).all(1).any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for run in [step] * 10 + [graph.replay] * 10:
        seen.zero_()
        seen_late.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            run()
        st.synchronize()
        assert torch.equal(out, want) and torch.equal(seen, want) and torch.equal(seen_late, want)

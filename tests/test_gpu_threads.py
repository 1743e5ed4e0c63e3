"""GPU: calls of one operator from several host threads (threads_client.cpp), each with its own batch, stream and sizes: every
call goes through and gives what it gives alone."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import test_gpu_adjust_logits as A
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
P, TIMES = ctypes.c_void_p, 10000


class Call(ctypes.Structure):  # AdjustCall and SampleCall
    _fields_ = [("meta", P), ("logits", P), ("how", P), ("out", P), ("stream", P), ("stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("vocab", ctypes.c_int32)]


@pytest.fixture(scope="module")
def client(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    lib = str(tmp_path_factory.mktemp("threads") / "libthreads.so")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-pthread", "-I", os.path.join(HERE, "..", "include"),
                        os.path.join(HERE, "threads_client.cpp"), "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return ctypes.CDLL(lib)


def together(run, fn, calls):
    """How many of the calls failed, each made TIMES times by a thread of its own."""
    return run(ctypes.cast(fn, P), (Call * len(calls))(*calls), len(calls), TIMES)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_rules_of_small_and_large_batches(client, dtype):
    # slices of 2048 tokens for the small ones, of 16384 for the large ones
    calls, keep, kind = [], [], R.DS_FP32 if dtype == "fp32" else R.DS_BF16
    for rows, vocab in ((1, 2000), (40, 131072), (1, 3000), (48, 120000)):
        st = torch.cuda.Stream()
        _, x = A.logits(rows, vocab, dtype)
        d, layer, out = A.made(rows, vocab, seed=vocab), A.meta_for(rows, st), torch.zeros_like(x)
        rules = A.given(d)
        calls.append(Call(ctypes.addressof(layer.meta), x.data_ptr(), ctypes.addressof(rules), out.data_ptr(), st.cuda_stream, vocab, kind, vocab))
        keep.append((x, out, d, layer, rules, st))
    torch.cuda.synchronize()
    assert together(client.adjust_together, R.load().ds_ragged_adjust_logits, calls) == 0
    torch.cuda.synchronize()
    for x, out, d, *_ in keep:
        A.holds(x, out, d)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_draws_of_small_and_large_vocabularies(client, dtype):
    calls, keep, kind = [], [], R.DS_FP32 if dtype == "fp32" else R.DS_BF16
    size = 4 if dtype == "fp32" else 2
    for rows, nbytes in ((200, 20000), (200, 66000), (200, 40000), (200, 120000)):  # of a row: 1 or 2 CTAs of different sizes
        st, vocab = torch.cuda.Stream(), nbytes // size
        _, x = A.logits(rows, vocab, dtype)
        layer, tokens = A.meta_for(rows, st), torch.zeros(rows, dtype=torch.int32, device="cuda")
        sampler = R.make_sampler(torch.rand(rows, device="cuda"))
        torch.cuda.synchronize()
        R.ds_ragged_sample(layer.meta, x, sampler, tokens, stream=st)
        calls.append(Call(ctypes.addressof(layer.meta), x.data_ptr(), ctypes.addressof(sampler), tokens.data_ptr(), st.cuda_stream, vocab, kind, vocab))
        torch.cuda.synchronize()
        keep.append((tokens, tokens.clone(), layer, sampler, x, st))
    assert together(client.sample_together, R.load().ds_ragged_sample, calls) == 0
    torch.cuda.synchronize()
    for tokens, want, *_ in keep:
        assert torch.equal(tokens, want)

"""GPU: ds_ragged_lora against out = base + scale B (A x) in 64 bits.

Tolerance, derived, with X = sum |a x| of an element of v = A x: a warp's chain
of tensor-core sums is at most in/128 + 32 long, each step within 2^-22 of X;
v reaches the second product within 2^-17 of itself (bf16: two 8-bit pieces),
or 2^-23 of the row's largest element (fp16: pieces of a scaled row, the second
maybe subnormal); the second product's sums are within (rank + 8) 2^-22; the
result is rounded once: finfo.eps/2 of it, and 2^-25 for fp16 subnormals.
"""
import numpy as np
import pytest
import torch

from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(new, which, n_adapters, rank, wi, wo, dtype, seed=0, pad=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = int(sum(new))
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    d = dict(new=np.array(new, np.int32), which=np.array(which, np.int32), na=n_adapters)
    d["x"] = (rand(n, wi + pad) * size).to(DT[dtype])[:, :wi]
    d["base"] = rand(n, wo + pad).to(DT[dtype])[:, :wo]
    d["a"] = (rand(n_adapters, rank, wi) / wi ** 0.5).to(DT[dtype])
    d["b"] = (rand(n_adapters, wo, rank) / rank ** 0.5 / size).to(DT[dtype])
    d["scale"] = 0.5 + torch.rand(n_adapters, generator=g, device="cuda")
    return d


def formula(d):
    """(out, tolerance) in 64 bits."""
    x, out = d["x"].double(), d["base"].double().clone()
    eps = torch.finfo(d["x"].dtype).eps
    tol = torch.full_like(out, 2.0 ** -25)
    token = torch.as_tensor(np.repeat(d["which"], d["new"]).astype(np.int64), device="cuda")
    wi, rank = d["a"].shape[2], d["a"].shape[1]
    for a in range(d["na"]):
        t = torch.nonzero(token == a)[:, 0]
        if not len(t):
            continue
        A, B = d["a"][a].double(), d["b"][a].double()
        s = float(d["scale"][a]) if d["scale"] is not None else 1.0
        v, mag = x[t] @ A.T, x[t].abs() @ A.abs().T
        off = mag * ((wi / 128 + 32) * 2.0 ** -22) + v.abs() * (2.0 ** -17 + (rank + 8) * 2.0 ** -22)
        off += v.abs().amax(1, keepdim=True) * 2.0 ** -23
        out[t] += s * (v @ B.T)
        tol[t] += s * (off @ B.abs().T)
    return out, tol + out.abs() * (eps / 2 + 2.0 ** -23)


def run(d, out=None, stream=None, plan=None):
    if plan is None:
        plan = R.LoraPlan(max(len(d["new"]), 1), max(int(d["new"].sum()), 1), stream=stream)
    plan.build(d["new"], d["which"], d["na"])
    if out is None:
        out = torch.full_like(d["base"], 7.0)
    R.ds_ragged_lora(plan.plan, R.make_lora(d["a"], d["b"], d["scale"]), d["x"], d["base"], out, stream)
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    return out


def check(d, **kw):
    want, tol = formula(d)
    base = d["base"].clone()
    out = run(d, **kw)
    bad = (out.double() - want).abs() > tol
    assert not bad.any(), "%d of %d off, rows %s" % (bad.sum(), bad.numel(), torch.nonzero(bad.any(1))[:8, 0].tolist())
    bare = torch.as_tensor(np.repeat(d["which"], d["new"]) < 0, device="cuda")
    assert torch.equal(out[bare], base[bare])
    return out


GROUPS = ([1, 15, 16, 17, 32, 33, 64, 65, 130, 1, 1, 2], [0, 1, 2, 3, 4, 5, 6, 7, 0, -1, 2, -1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("wi,wo", [(8, 8), (40, 520), (1000, 72), (4096, 1032)])
def test_matches_formula(wi, wo, rank, dtype):
    check(make(*GROUPS, 8, rank, wi, wo, dtype, seed=rank + wi))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,which,na", [
    ([1], [0], 1), ([1], [2], 3), ([1] * 256, list(range(256)), 256), ([1] * 40, [i % 3 - 1 for i in range(40)], 2),
    ([700], [0], 1), ([1, 300, 1, 300], [1, 0, 0, 1], 2), ([5, 6], [-1, -1], 2), ([33, 40, 300], [1, -1, -1], 2),
], ids=["one", "one_of_three", "all_different", "shared", "prompt", "split_groups", "bare", "bare_large"])
def test_batches(new, which, na, dtype):
    check(make(new, which, na, 16, 512, 768, dtype, seed=1))


@pytest.mark.parametrize("rank", [8, 16, 48, 64, 80, 128])
@pytest.mark.parametrize("wi,wo", [(8, 16), (64, 64), (200, 1000), (512, 320), (2048, 192)])
def test_large_tiles_of_every_cluster_size(wi, wo, rank):
    """Few, some and many tiles of up to 128 tokens: clusters of 8, 4, 2 and 1."""
    for tiles in (1, 40, 80, 160):
        new = [128] * (tiles - 1) + [100]
        check(make(new, list(range(tiles)), tiles, rank, wi, wo, "bf16" if tiles % 3 else "fp16", seed=tiles))


def test_rows_apart_in_place_and_behind_the_batch():
    d = make(*GROUPS, 8, 32, 256, 264, "bf16", seed=3, pad=24)
    n = d["base"].shape[0]
    want = check(d)
    store = torch.full((n + 3, 264 + 40), 5.0, dtype=torch.bfloat16, device="cuda")
    out = store[:, :264]
    d2 = dict(d)
    run(d2, out=out)
    assert torch.equal(out[:n], want) and (store[n:] == 5).all() and (store[:, 264:] == 5).all()
    d["base"] = d["base"].clone()
    run(d, out=d["base"])  # in place
    assert torch.equal(d["base"], want)


def test_no_scale_and_the_same_bits_again():
    d = make(*GROUPS, 8, 64, 1024, 512, "fp16", seed=4)
    d["scale"] = None
    a = check(d)
    for _ in range(3):
        assert torch.equal(run(d), a)


def test_large_intermediate_values_of_fp16():
    """A x beyond fp16's range, brought back by small B."""
    d = make([3, 70], [0, 1], 2, 16, 2048, 256, "fp16", seed=5, size=1e4)
    d["a"] *= 40
    assert torch.isfinite(d["x"]).all()
    assert (d["x"].double() @ d["a"][0].double().T).abs().max() > 2e5
    assert torch.isfinite(check(d)).all()


def test_infinities_and_nan_stay_in_their_row():
    d = make([1, 1, 40, 20], [0, 0, 1, -1], 2, 16, 512, 256, "bf16", seed=6)
    clean = run(d)
    d["x"][1, 3] = float("inf")
    d["x"][9, 0] = float("nan")
    d["x"][50, 0] = float("nan")  # a row without an adapter
    out = run(d)
    rest = torch.ones(62, dtype=torch.bool, device="cuda")
    rest[[1, 9]] = False
    assert torch.equal(out[rest], clean[rest])
    assert not torch.isfinite(out[1]).all() and torch.isnan(out[9]).all()


def test_a_server_without_adapters():
    d = make([3, 50, 1], [-1, -1, -1], 0, 16, 128, 192, "bf16", seed=8)
    out = torch.full_like(d["base"], 7.0)
    assert torch.equal(run(d, out=out), d["base"])
    keep = d["base"].clone()
    assert torch.equal(run(d, out=d["base"]), keep)  # in place: nothing to do


def test_one_short_and_one_long_sequence_of_each_length_around_a_run():
    for n in (31, 32, 33, 63, 64, 65, 127, 128, 129):
        check(make([n, 2, n], [1, 0, 1], 2, 16, 320, 136, "fp16", seed=n))


def test_empty_batch():
    d = make([], [], 1, 16, 64, 64, "bf16")
    out = torch.full((1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    d["x"], d["base"] = torch.zeros_like(out), torch.zeros_like(out)
    assert (run(d, out=out) == 3).all()


def test_a_call_that_reads_what_the_last_one_wrote():
    """Both launches of a call are complete before what follows on the stream reads its rows."""
    d = make([1] * 60 + [700, 90, 33], [i % 8 for i in range(63)], 8, 32, 512, 512, "bf16", seed=9)
    lora = R.make_lora(d["a"], d["b"] * 0.1, d["scale"])
    plan = R.LoraPlan(63, int(d["new"].sum()))
    plan.build(d["new"], d["which"], 8)
    want = [d["x"]]
    for _ in range(4):
        want.append(torch.empty_like(d["base"]))
        R.ds_ragged_lora(plan.plan, lora, want[-2], d["base"], want[-1])
        torch.cuda.synchronize()
    for _ in range(40):
        got = [d["x"]] + [torch.zeros_like(d["base"]) for _ in range(4)]
        last = torch.empty_like(d["base"])
        for a, b in zip(got, got[1:]):
            R.ds_ragged_lora(plan.plan, lora, a, d["base"], b, torch.cuda.current_stream())
        last.copy_(got[-1])
        assert torch.equal(last, want[-1])


def test_streams_and_a_captured_call_for_other_batches():
    st = torch.cuda.Stream()
    d = make(*GROUPS, 8, 16, 512, 320, "bf16", seed=7)
    lora = R.make_lora(d["a"], d["b"], d["scale"])
    torch.cuda.synchronize()
    plan = R.LoraPlan(16, 400, stream=st, flags=R.DS_META_CAPACITY)
    rows = 400 - d["x"].shape[0]
    d["x"], d["base"] = (torch.cat([v, v[:rows]]) for v in (d["x"], d["base"]))
    out = torch.zeros_like(d["base"])
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        plan.build(d["new"], d["which"], 8)
        R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out, st)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        plan.build(d["new"], d["which"], 8)
        R.ds_ragged_lora(plan.plan, lora, d["x"], d["base"], out, st)
    for new, which in (([1], [3]), ([], []), GROUPS, ([40, 1, 1, 300], [0, 5, -1, 0]), ([1] * 16, list(range(8)) * 2)):
        n = sum(new)
        plan.pack(new, which, 8)
        out.fill_(9)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        st.synchronize()
        part = dict(d, new=np.array(new, int), which=np.array(which, int), x=d["x"][:n], base=d["base"][:n])
        want, tol = formula(part)
        assert ((out[:n].double() - want).abs() <= tol).all() and (out[n:] == 9).all()

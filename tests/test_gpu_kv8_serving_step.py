"""GPU: the calls on the 8-bit pool and the rules on logits together, as a server runs
them: embedding, projection, append to the 8-bit pool, attention over it, output
projection, last-token rows, the requests' rules, draw; then the drawn tokens as the
next step, in the requests' histories.

Each stage is held to its definition on what the stage before it gave (the stages' own
tolerances); a captured step gives the same bits as an eager one.
"""
import numpy as np
import pytest
import torch

import kv8_formula as K
import test_gpu_adjust_logits as J
import test_gpu_kv8_append as A
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HIDDEN, VOCAB, ROOM = 256, 1003, 400


class Model:
    def __init__(self, heads, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.d = heads
        dt = J.DT[dtype]
        rand = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(dt)  # noqa: E731
        width = (self.hq + 2 * self.hkv) * self.d
        self.table, self.head = rand(VOCAB + 5, HIDDEN), rand(HIDDEN, VOCAB, k=0.2)
        self.wqkv, self.wo = rand(HIDDEN, width, k=HIDDEN ** -0.5), rand(self.hq * self.d, HIDDEN, k=0.06)


class State:
    """Buffers of a step for up to `seqs` sequences and `tokens` tokens."""

    def __init__(self, m, wl, st, seqs, tokens, flags, rules, sampler):
        dev, dt = "cuda", W.torch_dtype(wl)
        self.layer = R.RaggedLayer(R.params_for(wl), seqs, tokens, 128, ROOM, stream=st, flags=flags)
        self.ids = torch.zeros(tokens, dtype=torch.int32, device=dev)
        self.x, self.att = torch.zeros((tokens, HIDDEN), dtype=dt, device=dev), torch.zeros((tokens, m.hq * m.d), dtype=dt, device=dev)
        self.qkv = torch.zeros((tokens, (m.hq + 2 * m.hkv) * m.d), dtype=dt, device=dev)
        self.hidden, self.rows = torch.zeros((tokens, HIDDEN), dtype=dt, device=dev), torch.zeros((seqs, HIDDEN), dtype=dt, device=dev)
        self.logits, self.ruled = (torch.zeros((seqs, VOCAB), dtype=dt, device=dev) for _ in range(2))
        self.tokens = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.m, self.st, self.rules, self.sampler = m, st, rules, sampler

    def step(self, descs, blocks, pool):
        m, meta = self.m, self.layer.meta
        self.layer.build(descs, blocks)
        R.ds_ragged_embedding(meta, self.ids, m.table, self.x, self.st)
        torch.matmul(self.x, m.wqkv, out=self.qkv)
        self.layer.append8(self.qkv, pool)
        self.layer.attention8(self.qkv, pool, self.att)
        torch.matmul(self.att, m.wo, out=self.hidden)
        R.ds_ragged_logits_gather(meta, self.hidden, self.rows, self.st)
        torch.matmul(self.rows, m.head, out=self.logits)
        R.ds_ragged_adjust_logits(meta, self.logits, self.rules, self.ruled, self.st)
        R.ds_ragged_sample(meta, self.ruled, self.sampler, self.tokens, None, self.st)


@pytest.mark.parametrize("heads,dtype", [((4, 2, 64), "fp16"), ((8, 1, 128), "bf16")])
def test_steps_of_a_mixed_batch(heads, dtype):
    m = Model(heads, dtype)
    seqs = [(0, 40), (70, 1), (63, 1), (0, 1), (10, 33), (128, 3)]
    n = len(seqs)
    g = torch.Generator(device="cuda").manual_seed(7)
    plan = W.make_custom([(s + c + 2, 2) for s, c in seqs], *heads, dtype=dtype, seed=3)  # blocks for four steps
    seen, new = np.array([s for s, _ in seqs]), np.array([c for _, c in seqs])

    def batch():
        wl = W.make_custom(list(zip(seen.tolist(), new.tolist())), *heads, dtype=dtype, seed=3)
        wl.block_ids, wl.num_blocks = plan.block_ids, plan.num_blocks
        return wl

    codes, scales = K.blanked(batch(), *K.made_pool(batch(), 1))
    rules = J.made(n, VOCAB, seed=4, history=60)
    rules["history_len"] = np.minimum(rules["history_len"], 50).astype(np.int32)
    rules["mask_row"] = np.array([1, 2, -1, 1, 2, 1], np.int32)  # none without a token
    t = {k: torch.as_tensor(v).cuda().contiguous() for k, v in rules.items()}
    handle = R.make_logit_rules(**t)
    sampler = R.make_sampler(torch.rand(n, generator=g, device="cuda"), torch.tensor([0.8, 1.0, 0.0, 1.2, 0.7, 1.0], device="cuda"))
    st = torch.cuda.Stream()
    eager, cap = State(m, batch(), st, n, int(new.sum()), 0, handle, sampler), State(m, batch(), st, n, 96, R.DS_META_CAPACITY, handle, sampler)
    first = torch.randint(0, VOCAB, (int(new.sum()),), generator=g, device="cuda", dtype=torch.int32)
    eager.ids[:] = first
    other = (codes.clone(), scales.clone())
    pool, pool2 = R.make_kv8_pool(codes, scales), R.make_kv8_pool(*other)
    torch.cuda.synchronize()
    graph = None
    for step in range(4):
        wl = batch()
        descs = R.SeqDescs.of(wl)
        before = (codes.clone(), scales.clone())
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            eager.step(descs, wl.num_blocks, pool)
        st.synchronize()
        assert eager.layer.device_error() == 0
        c = int(new.sum())
        A.check(wl, eager.qkv, before, (codes, scales))
        K.holds(wl, eager.att, eager.qkv, codes, scales)
        J.holds(eager.logits, eager.ruled, {k: v.cpu().numpy() for k, v in t.items()})
        drawn = eager.tokens.clone()
        assert (drawn >= 0).all() and not torch.isneginf(eager.ruled.gather(1, drawn[:, None].long())).any()
        # the same step captured, in launches for the capacities
        cap.ids[:c] = eager.ids[:c]
        torch.cuda.synchronize()
        if graph is None:
            saved = (other[0].clone(), other[1].clone())
            with torch.cuda.stream(st):
                cap.step(descs, wl.num_blocks, pool2)  # the libraries' own warm-up
            st.synchronize()
            other[0].copy_(saved[0]), other[1].copy_(saved[1])
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                cap.step(descs, wl.num_blocks, pool2)
        cap.layer.pack(descs, wl.num_blocks)
        with torch.cuda.stream(st):
            graph.replay()
        st.synchronize()
        assert cap.layer.device_error() == 0
        assert torch.equal(cap.qkv[:c], eager.qkv[:c])
        assert torch.equal(other[1].nan_to_num(), scales.nan_to_num()) and A.same_codes(other[0], codes)
        K.holds(wl, cap.att, cap.qkv, codes, scales)
        # the drawn tokens come next, and into the histories
        seen, new = seen + new, np.ones(n, np.int64)
        if step == 0:
            eager = State(m, batch(), st, n, n, 0, handle, sampler)
        eager.ids[:n] = drawn
        t["history"].scatter_(1, t["history_len"].long()[:, None], drawn[:, None])
        t["history_len"] += 1
        torch.cuda.synchronize()

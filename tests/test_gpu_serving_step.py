"""GPU: the operators of one serving step together, as a server runs them: embedding,
adapted qkv projection, norm + rotation + append, blocked attention, adapted
output projection, last-token rows, draw; then the drawn tokens as the next step.

Each stage is held to its formula in 64 bits on what the stage before it gave
(the stages' own tolerances); a captured step gives the same bits as an eager one.
"""
import numpy as np
import pytest
import torch

import test_gpu_lora as L
import test_gpu_norm_append as A
import test_gpu_sample as S
from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
from ragged_blocked_kv_raggedbatch_gb300 import workloads as W

pytestmark = pytest.mark.gpu

HQ, HKV, D, HIDDEN, VOCAB, RANK = 4, 2, 64, 256, 1003, 16


class Model:
    def __init__(self, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = L.DT[dtype]
        rand = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(dt)  # noqa: E731
        width = (HQ + 2 * HKV) * D
        self.dtype, self.dt = dtype, dt
        self.table, self.head = rand(VOCAB + 5, HIDDEN), rand(HIDDEN, VOCAB, k=0.2)
        self.wqkv, self.wo = rand(HIDDEN, width, k=HIDDEN ** -0.5), rand(HQ * D, HIDDEN, k=0.06)
        self.a1, self.b1 = rand(3, RANK, HIDDEN, k=HIDDEN ** -0.5), rand(3, width, RANK, k=RANK ** -0.5)
        self.a2, self.b2 = rand(3, RANK, HQ * D, k=0.06), rand(3, HIDDEN, RANK, k=RANK ** -0.5)
        self.scale = 0.5 + torch.rand(3, generator=g, device="cuda")
        self.norm = R.make_qk_norm(1 + rand(D, k=0.1), 1 + rand(D, k=0.1))
        self.lora1, self.lora2 = R.make_lora(self.a1, self.b1, self.scale), R.make_lora(self.a2, self.b2, self.scale)


def attend(m, wl, q, pool):
    """Causal attention in 64 bits of normalised, unrotated queries over the pool's keys and values."""
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(wl.seen, wl.new)])
    f = (np.float64(np.float32(wl.rope_theta)) ** (-2.0 * np.arange(D // 2) / D)).astype(np.float32)
    ang = torch.as_tensor((pos.astype(np.float32)[:, None] * f).astype(np.float64)[:, None], device="cuda")
    q = q.double().view(-1, HQ, D)
    a, b = q[..., :D // 2], q[..., D // 2:]
    q = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    out, at = torch.empty_like(q), 0
    for i in range(wl.n_seqs):
        ids = torch.as_tensor(np.asarray(wl.block_ids[i]), device="cuda").long()
        kv = pool[ids].double().permute(1, 2, 0, 3, 4).reshape(2, HKV, -1, D).repeat_interleave(HQ // HKV, 1)
        for j in range(int(wl.new[i])):
            n = int(wl.seen[i]) + j + 1
            p = torch.softmax((kv[0, :, :n] @ q[at + j][:, :, None])[..., 0] * D ** -0.5, -1)
            out[at + j] = (p[:, None] @ kv[1, :, :n])[:, 0]
        at += int(wl.new[i])
    return out.view(-1, HQ * D)


def lora_holds(out, base, x, a, b, scale, new, which):
    d = dict(x=x, base=base, a=a, b=b, scale=scale, na=3, new=np.asarray(new), which=np.asarray(which))
    want, tol = L.formula(d)
    assert ((out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_steps_of_a_mixed_batch(dtype):
    m = Model(dtype)
    seqs, which = [(0, 40), (70, 1), (63, 1), (0, 1), (10, 33), (128, 3)], [0, 1, -1, 2, 2, 0]
    g = torch.Generator(device="cuda").manual_seed(7)
    wl = W.make_custom([(s + n, 2) for s, n in seqs], HQ, HKV, D, dtype=dtype, seed=3)  # blocks for two steps
    pool = torch.randn(wl.pool_shape(), generator=g, device="cuda").to(m.dt)
    seen, new = np.array([s for s, _ in seqs], np.int32), np.array([n for _, n in seqs], np.int32)
    ids = torch.randint(0, VOCAB, (int(new.sum()),), generator=g, device="cuda", dtype=torch.int32)
    n_seqs = len(seqs)
    sp = R.make_sampler(torch.rand(n_seqs, generator=g, device="cuda"), torch.tensor([0.8, 1.0, 0.0, 1.2, 0.7, 1.0], device="cuda"),
                        torch.tensor([0, 20, 0, 5, 300, 0], device="cuda", dtype=torch.int32),
                        torch.tensor([0.9, 1.0, 1.0, 0.8, 0.95, 1.0], device="cuda"), torch.tensor([0.0, 0.05, 0, 0, 0, 0.1], device="cuda"))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for step in range(2):
        wl.seen, wl.new = seen, new
        n = int(new.sum())
        e = lambda rows, cols, dt=m.dt: torch.zeros((rows, cols), dtype=dt, device="cuda")  # noqa: E731
        x, qkv, att, y, last = e(n, HIDDEN), e(n, (HQ + 2 * HKV) * D), e(n, HQ * D), e(n, HIDDEN), e(n_seqs, HIDDEN)
        base1, base2 = torch.empty_like(qkv), torch.empty_like(y)
        tok, lp, logits = torch.zeros(n_seqs, dtype=torch.int32, device="cuda"), torch.zeros(n_seqs, device="cuda"), e(n_seqs, VOCAB)
        layer = R.RaggedLayer(R.params_for(wl), n_seqs, n, int(wl.blocks_needed().sum()), wl.max_len(), stream=st)
        plan = R.LoraPlan(n_seqs, n, stream=st)
        torch.cuda.synchronize()

        def run(p):
            layer.build(R.SeqDescs.of(wl), wl.num_blocks)
            plan.build(new, which, 3)
            R.ds_ragged_embedding(layer.meta, ids, m.table, x, st)
            torch.matmul(x, m.wqkv, out=base1)
            R.ds_ragged_lora(plan.plan, m.lora1, x, base1, qkv, st)
            layer.norm_append(m.norm, qkv, p, qkv_out=qkv)
            layer.attention(qkv, p, att)
            torch.matmul(att, m.wo, out=base2)
            R.ds_ragged_lora(plan.plan, m.lora2, att, base2, y, st)
            R.ds_ragged_logits_gather(layer.meta, y, last, st)
            torch.matmul(last, m.head, out=logits)
            R.ds_ragged_sample(layer.meta, logits, sp, tok, lp, st)

        before, graphed = pool.clone(), pool.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            run(pool)
        st.synchronize()
        assert layer.device_error() == 0 and plan.device_error() == 0
        assert torch.equal(x, m.table[ids.long()])
        raw = torch.empty_like(qkv)
        with torch.cuda.stream(st):  # the qkv rows before their queries were replaced in place
            R.ds_ragged_lora(plan.plan, m.lora1, x, base1, raw, st)
        st.synchronize()
        lora_holds(raw, base1, x, m.a1, m.b1, m.scale, new, which)
        nq, _, yk, v, _, sk = A.formula(wl, raw, *m.norm.tensors, np.float32(1e-6), R.DS_ROPE_HALF)
        A.close(qkv[:, :HQ * D], nq, np.abs(nq), wl)
        A.check_pool(wl, before, pool, yk, v, sk)
        off = (att.double() - attend(m, wl, qkv[:, :HQ * D], pool)).abs().max()
        assert off <= {"fp16": 1e-2, "bf16": 2e-2}[dtype], off  # the attention call's stated bar
        lora_holds(y, base2, att, m.a2, m.b2, m.scale, new, which)
        ends = np.cumsum(new) - 1
        assert torch.equal(last, y[torch.as_tensor(ends, device="cuda")])
        kw = {k: sp.tensors[k].double().cpu().numpy() for k in sp.tensors}
        for i in range(n_seqs):
            want, wlp = S.one_row(logits[i].double().cpu().numpy(), kw["uniforms"][i], kw["temperature"][i], int(kw["top_k"][i]),
                                  kw["top_p"][i], kw["min_p"][i])
            assert int(tok[i]) == want and abs(float(lp[i]) - wlp) <= 2.0 ** -24 * abs(wlp) + 1e-9
        eager = [t.clone() for t in (pool, att, y, tok, lp)]
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            run(graphed)
        tok.fill_(-5)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            gr.replay()
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, (graphed, att, y, tok, lp)))
        seen, new = seen + new, np.ones(n_seqs, np.int32)
        ids = tok.clone()

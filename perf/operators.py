"""Timed cases of three operators around the attention call of a ragged batch.

  append  per-head RMS norm of queries and keys, position rotation, and the append of keys and
          values to the blocked KV pool, in one pass (``ds_kv_norm_rotary_append``)
  lora    low-rank adapters, one per sequence of the batch, added to a shared projection's
          output (``ds_ragged_lora``)
  sample  one token for each sequence from its logits row: temperature, top-k, top-p and min-p,
          from a given uniform number (``ds_ragged_sample``)

``run`` computes them in elementary torch operations, or, with ``own`` set, through the calls
that a user of the package makes.  ``exact`` computes the same from the definitions in 64 bits.

Definitions.
  append: for a query or key head x of a packed token at position p,
          n = x * w / sqrt(mean(x^2) + eps), then each pair (n0, n1) of the rotary pairing turns by
          the angle a = fp32(fp32(p) * fp32(theta^(-2k/d))): (n0 cos a - n1 sin a, n1 cos a + n0 sin a).
          Keys go to the pool rotated, values as they are; normalised queries are returned unrotated
          (the attention call rotates them on load), and rotated where a case asks for it.
  lora:   out[t] = base[t] + scale_a * B_a (A_a x[t]) with a the adapter of token t's sequence;
          out[t] = base[t] where the sequence has none.
  sample: tokens in descending order of their logit, the lower index first among equals; weights
          w = exp((x - max) / T); kept are the first top_k tokens, of those the shortest run of
          leading ones that holds top_p of their weight, of those the ones with w >= min_p; chosen
          is the first kept token, by index, whose running sum of weights passes u times the kept weight.
          T = 0 takes the first token; its log-probability is 0.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 64
DEV = "cuda"

# (query heads, KV heads, head_dim) of the workloads, and small ones
HEADS = [(32, 32, 128), (32, 8, 128), (64, 8, 128), (4, 2, 64), (16, 2, 128), (8, 4, 64)]


def listed():
    return [
        # one request generating alone: the call's latency
        dict(name="append_1_token", op="append", decodes=1, chunks=0, tokens=0, max_seen=4000, heads="32,8,128",
             dtype="bf16", style="half", theta=5.0e5, per_head=False, rotated=False),
        # a full decode-only batch with one KV head per query head
        dict(name="append_256_decodes", op="append", decodes=256, chunks=0, tokens=0, max_seen=127, heads="32,32,128",
             dtype="bf16", style="half", theta=1.0e4, per_head=False, rotated=False),
        # a mixed batch: prompt chunks and decodes, a weight for each head, adjacent pairs, small heads
        dict(name="append_mixed_small_heads", op="append", decodes=61, chunks=5, tokens=1234, max_seen=900, heads="8,4,64",
             dtype="fp16", style="interleaved", theta=1.0e4, per_head=True, rotated=True),
        # two long prompt chunks of a large grouped-query layer
        dict(name="append_2x8192", op="append", decodes=0, chunks=2, tokens=16384, max_seen=4096, heads="64,8,128",
             dtype="bf16", style="half", theta=5.0e5, per_head=False, rotated=False),
        # one request with its adapter on the query/key/value projection
        dict(name="lora_1_token", op="lora", decodes=1, chunks=0, tokens=0, adapters=4, bare=0, rank=16, width_in=4096,
             width_out=6144, dtype="bf16"),
        # a decode-only batch of 256 requests over 64 adapters
        dict(name="lora_256_decodes_64_adapters", op="lora", decodes=256, chunks=0, tokens=0, adapters=64, bare=0, rank=16,
             width_in=4096, width_out=6144, dtype="bf16"),
        # prompt chunks beside decodes, some requests without an adapter, on the output projection
        dict(name="lora_mixed_2048", op="lora", decodes=512, chunks=3, tokens=1536, adapters=16, bare=40, rank=32,
             width_in=4096, width_out=4096, dtype="fp16"),
        # a full batch of prompt chunks with a large rank
        dict(name="lora_8192_prompts", op="lora", decodes=0, chunks=16, tokens=8192, adapters=8, bare=0, rank=64, width_in=4096,
             width_out=6144, dtype="bf16"),
        # one request: latency of a draw with top-p from 32-bit logits
        dict(name="sample_1_row", op="sample", rows=1, vocab=32000, dtype="fp32", mode="top_p", banned=0.0),
        # a batch in which each request has its own settings
        dict(name="sample_256_mixed", op="sample", rows=256, vocab=131072, dtype="bf16", mode="mixed", banned=0.0),
        # an odd vocabulary (rows that start anywhere), a grammar's mask, top-k with min-p
        dict(name="sample_64_top_k_masked", op="sample", rows=64, vocab=50001, dtype="fp16", mode="top_k", banned=0.6),
        # temperature alone from 32-bit logits: every token counts
        dict(name="sample_256_temperature", op="sample", rows=256, vocab=131072, dtype="fp32", mode="temperature", banned=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "lora", "sample"])
    kind = rng.choice(["decode", "prompt", "mixed"])
    c = {"op": op}
    if op == "sample":
        c.update(rows=_log_int(rng, 1, 256), vocab=_log_int(rng, 500, 131072), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                 mode=rng.choice(["mixed", "top_p", "top_k", "temperature", "min_p"]), banned=rng.choice([0.0, 0.0, 0.6]))
        return c
    c["decodes"] = 0 if kind == "prompt" else _log_int(rng, 1, 256)
    c["chunks"] = 0 if kind == "decode" else _log_int(rng, 1, 16)
    c["tokens"] = 0 if kind == "decode" else max(2 * c["chunks"], _log_int(rng, 16, 7900))
    if op == "append":
        c.update(max_seen=_log_int(rng, 1, 1500), dtype=rng.choice(["bf16", "fp16"]), style=rng.choice(["half", "interleaved"]),
                 theta=rng.choice([1.0e4, 5.0e5, 1.0e6]), per_head=rng.random() < 0.5, rotated=rng.random() < 0.5)
        c["heads"] = "%d,%d,%d" % rng.choice(HEADS)
        if c["heads"] == "32,32,128":
            c["max_seen"] = min(c["max_seen"], 127)
    else:
        seqs = c["decodes"] + c["chunks"]
        c.update(adapters=_log_int(rng, 1, 64), bare=rng.choice([0, 0, seqs // 5]), rank=8 * _log_int(rng, 1, 8),
                 width_in=8 * _log_int(rng, 64, 512), width_out=8 * _log_int(rng, 64, 768), dtype=rng.choice(["bf16", "fp16"]))
    return c


def _batch(case, rs):
    """(seen, new) of the batch's sequences, in a drawn order."""
    new = [1] * case["decodes"]
    if case["chunks"]:
        spare = case["tokens"] - 2 * case["chunks"]
        cuts = np.sort(rs.randint(0, spare + 1, case["chunks"] - 1))
        new += list(2 + np.diff(np.concatenate([[0], cuts, [spare]])))
    new = np.array(new, np.int32)[rs.permutation(len(new))]
    seen = rs.randint(0, case.get("max_seen", 0) + 1, len(new)).astype(np.int32)
    return seen, new


def _n_tokens(case):
    return case["decodes"] + (case["tokens"] if case["chunks"] else 0)


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _on(a, dtype=torch.int64):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device=DEV)


# ------------------------------------------------------------------ inputs --


def _prepare_append(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d = (int(v) for v in case["heads"].split(","))
    dt = DTYPES[case["dtype"]]
    seen, new = _batch(case, rs)
    total = seen.astype(np.int64) + new
    need = (total + BLOCK - 1) // BLOCK
    # the pool's size goes by the case alone: room for the longest histories the case can draw
    ids = rs.permutation(len(new) * (case["max_seen"] // BLOCK + 2) + int(new.sum()) // BLOCK).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    seq = np.repeat(np.arange(len(new)), new)
    first = np.concatenate([[0], np.cumsum(new)])[:-1]
    pos = seen[seq] + (np.arange(len(seq)) - first[seq])
    n, positions = len(seq), int(total.max())
    s = dict(case=case, hq=hq, hkv=hkv, d=d, eps=1e-6, n=n)
    s["qkv"] = _normal(gen, (n, (hq + 2 * hkv) * d), dt)
    s["q_weight"] = (1 + 0.2 * torch.randn((hq if case["per_head"] else 1, d), generator=gen, device=DEV)).to(dt)
    s["k_weight"] = (1 + 0.2 * torch.randn((hkv if case["per_head"] else 1, d), generator=gen, device=DEV)).to(dt)
    s["pool"] = _normal(gen, (1, 2, hkv, BLOCK, d), dt).repeat(len(ids), 1, 1, 1, 1)
    s["block"], s["slot"], s["pos"] = _on(ids[at[seq] + pos // BLOCK]), _on(pos % BLOCK), _on(pos)
    k = torch.arange(d // 2, device=DEV, dtype=torch.float64)
    turn = torch.arange(positions, device=DEV, dtype=torch.float32)[:, None] * torch.pow(torch.tensor(np.float32(case["theta"]), dtype=torch.float64, device=DEV), -2 * k / d).float()
    s["cos"], s["sin"] = torch.cos(turn.double()).float(), torch.sin(turn.double()).float()
    s["qkv_out"] = torch.zeros_like(s["qkv"])
    s["q_out"] = torch.zeros((n, hq * d), dtype=dt, device=DEV) if case["rotated"] else None
    if own:
        from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
        style = R.DS_ROPE_HALF if case["style"] == "half" else R.DS_ROPE_INTERLEAVED
        params = R.make_params(hq, hkv, d, case["dtype"], case["theta"], style)
        s["stream"] = torch.cuda.current_stream()
        s["layer"] = R.RaggedLayer(params, len(new), n, int(need.sum()), positions, stream=s["stream"])
        s["layer"].build(R.SeqDescs(seen, new, [ids[at[i]:at[i + 1]] for i in range(len(new))]), len(ids))
        s["norm"] = R.make_qk_norm(s["q_weight"], s["k_weight"], s["eps"], per_head=case["per_head"])
    return s


def _prepare_lora(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    seen, new = _batch(case, rs)
    which = rs.permutation(case["adapters"])[np.arange(len(new)) % case["adapters"]].astype(np.int32)
    which[rs.permutation(len(new))[:case["bare"]]] = -1
    n, r, wi, wo, na = int(new.sum()), case["rank"], case["width_in"], case["width_out"], case["adapters"]
    s = dict(case=case)
    s["x"] = _normal(gen, (n, wi), dt)
    s["base"] = _normal(gen, (n, wo), dt)
    s["a"] = _normal(gen, (na, r, wi), dt, 1 / math.sqrt(wi))
    s["b"] = _normal(gen, (na, wo, r), dt, 1 / math.sqrt(r))
    s["scale"] = 0.5 + torch.rand(na, generator=gen, device=DEV)
    s["token_adapter"] = _on(np.repeat(which, new))
    s["out"] = torch.zeros_like(s["base"])
    if own:
        from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
        s["stream"] = torch.cuda.current_stream()
        s["plan"] = R.LoraPlan(len(new), n, stream=s["stream"])
        s["plan"].build(new, which, na)
        s["lora"] = R.make_lora(s["a"], s["b"], s["scale"])
    return s


def _prepare_sample(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows, vocab, mode = case["rows"], case["vocab"], case["mode"]
    x = 2.2 * torch.randn((rows, vocab), generator=gen, device=DEV)
    # a few likely tokens stand out, as they do in a trained model's rows
    likely = torch.randint(0, vocab, (rows, 24), generator=gen, device=DEV)
    x.scatter_add_(1, likely, 9 * torch.rand((rows, 24), generator=gen, device=DEV))
    if case["banned"]:
        x.masked_fill_(torch.rand((rows, vocab), generator=gen, device=DEV) < case["banned"], -math.inf)
    s = dict(case=case, logits=x.to(DTYPES[case["dtype"]]))
    pick = lambda on, off: np.where(rs.rand(rows) < 0.6, on, off) if mode == "mixed" else on  # noqa: E731
    temperature = rs.uniform(0.5, 1.3, rows)
    if mode == "mixed":
        temperature = np.where(rs.rand(rows) < 0.1, 0.0, temperature)
    top_k = pick(np.exp(rs.uniform(math.log(5), math.log(400), rows)).astype(np.int32), 0) if mode in ("mixed", "top_k") else np.zeros(rows)
    top_p = pick(rs.uniform(0.7, 0.99, rows), 1.0) if mode in ("mixed", "top_p") else np.ones(rows)
    min_p = pick(rs.uniform(0.01, 0.2, rows), 0.0) if mode in ("mixed", "top_k", "min_p") else np.zeros(rows)
    s["temperature"], s["top_k"] = _on(temperature, torch.float32), _on(top_k, torch.int32)
    s["top_p"], s["min_p"] = _on(top_p, torch.float32), _on(min_p, torch.float32)
    s["uniforms"] = torch.rand(rows, generator=gen, device=DEV)
    s["tokens"] = torch.zeros(rows, dtype=torch.int32, device=DEV)
    s["logprobs"] = torch.zeros(rows, device=DEV)
    if own:
        from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
        s["stream"] = torch.cuda.current_stream()
        s["layer"] = R.RaggedLayer(R.make_params(1, 1, 64), rows, rows, rows, 1, stream=s["stream"])
        s["layer"].build(R.SeqDescs([0] * rows, [1] * rows, [np.array([i], np.int32) for i in range(rows)]), rows)
        s["sampler"] = R.make_sampler(s["uniforms"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    return s


def prepare(case, seed):
    return {"append": _prepare_append, "lora": _prepare_lora, "sample": _prepare_sample}[case["op"]](case, seed)


# -------------------------------------------------------------- plain forms --


def _turned(x, c, s, style):
    """x [n, heads, d], c and s [n, 1, d/2]: each pair of the pairing rotated."""
    half = x.shape[-1] // 2
    if style == "half":
        x0, x1 = x[..., :half], x[..., half:]
        return torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)


def _append(s):
    n, hq, hkv, d, dt, style = s["n"], s["hq"], s["hkv"], s["d"], s["qkv"].dtype, s["case"]["style"]
    x = s["qkv"].view(n, hq + 2 * hkv, d)
    q, k = x[:, :hq].float(), x[:, hq:hq + hkv].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + s["eps"]) * s["q_weight"].float()
    k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + s["eps"]) * s["k_weight"].float()
    c, t = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
    s["pool"][s["block"], 0, :, s["slot"]] = _turned(k, c, t, style).to(dt)
    s["pool"][s["block"], 1, :, s["slot"]] = x[:, hq + hkv:]
    got = {"pool": s["pool"], "queries": q.to(dt).view(n, hq * d)}
    if s["q_out"] is not None:
        got["rotated"] = _turned(q, c, t, style).to(dt).view(n, hq * d)
    return got


def _lora(s):
    na, r, wi = s["a"].shape
    mine = s["token_adapter"][:, None] == torch.arange(na, device=DEV)
    v = (s["x"].float() @ s["a"].float().view(na * r, wi).t()).view(-1, na, r)
    v = (v * (mine * s["scale"])[:, :, None]).view(-1, na * r)
    return {"out": (s["base"].float() + v @ s["b"].float().transpose(1, 2).reshape(na * r, -1)).to(s["base"].dtype)}


def _sample(s):
    x, at = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t, vocab = s["temperature"].double()[:, None], x.shape[1]
    place = torch.arange(vocab, device=DEV)
    w = torch.where(x == x[:, :1], 1.0, torch.exp((x - x[:, :1]) / torch.where(t > 0, t, 1.0)))
    k = s["top_k"].long()[:, None]
    w = torch.where((k > 0) & (place >= k) | (t <= 0) & (place > 0), 0.0, w)
    upto = torch.cumsum(w, 1)
    p = s["top_p"].double()[:, None]
    w = torch.where((p < 1) & (upto - w >= p * upto[:, -1:]) & (place > 0), 0.0, w)
    w = torch.where(w < s["min_p"].double()[:, None], 0.0, w)
    w = torch.zeros_like(w).scatter_(1, at, w)  # back in the tokens' own order
    upto = torch.cumsum(w, 1)
    mass = upto[:, -1:]
    chosen = (upto <= s["uniforms"].double()[:, None] * mass).sum(1, keepdim=True)
    return {"tokens": chosen[:, 0].int(), "logprobs": torch.log(w.gather(1, chosen) / mass)[:, 0].float()}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _append, "lora": _lora, "sample": _sample}[op](state)
    from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
    s = state
    if op == "append":
        s["layer"].norm_append(s["norm"], s["qkv"], s["pool"], qkv_out=s["qkv_out"], q_out=s["q_out"])
        got = {"pool": s["pool"], "queries": s["qkv_out"][:, :s["hq"] * s["d"]]}
        if s["q_out"] is not None:
            got["rotated"] = s["q_out"]
        return got
    if op == "lora":
        R.ds_ragged_lora(s["plan"].plan, s["lora"], s["x"], s["base"], s["out"], s["stream"])
        return {"out": s["out"]}
    R.ds_ragged_sample(s["layer"].meta, s["logits"], s["sampler"], s["tokens"], s["logprobs"], s["stream"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


# ------------------------------------------------------- 64-bit definitions --


def _exact_append(case, s):
    hq, hkv, d, n = s["hq"], s["hkv"], s["d"], s["n"]
    x = s["qkv"].double().reshape(n, -1, d)
    freq = np.float32(np.float64(np.float32(case["theta"])) ** (-2.0 * np.arange(d // 2) / d))
    angle = s["pos"].cpu().numpy().astype(np.float32)[:, None] * freq[None, :]
    angle = torch.as_tensor(angle.astype(np.float64), device=DEV)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    pair = (lambda v: v.reshape(n, -1, 2, d // 2).transpose(-1, -2)) if case["style"] == "half" else (lambda v: v.reshape(n, -1, d // 2, 2))

    def normed(v, w):
        return v / torch.sqrt((v * v).sum(-1, keepdim=True) / d + s["eps"]) * w.double()

    def turned(v):
        z = torch.view_as_real(torch.view_as_complex(pair(v).contiguous()) * turn)
        return (z.transpose(-1, -2) if case["style"] == "half" else z).reshape(n, -1, d)

    q, k = normed(x[:, :hq], s["q_weight"]), normed(x[:, hq:hq + hkv], s["k_weight"])
    pool = s["pool"].double()
    both = torch.stack([turned(k), x[:, hq + hkv:]], 1)
    pool.permute(0, 3, 1, 2, 4)[s["block"], s["slot"]] = both
    got = {"pool": pool, "queries": q.reshape(n, -1)}
    if case["rotated"]:
        got["rotated"] = turned(q).reshape(n, -1)
    return got


def _exact_lora(case, s):
    out = s["base"].double()
    for a in range(case["adapters"]):
        t = torch.nonzero(s["token_adapter"] == a)[:, 0]
        v = torch.einsum("th,rh->tr", s["x"][t].double(), s["a"][a].double())
        out[t] += float(s["scale"][a]) * torch.einsum("tr,or->to", v, s["b"][a].double())
    return {"out": out}


def _exact_sample(case, s):
    x = s["logits"].double().cpu().numpy()
    v = {k: s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p", "min_p", "uniforms")}
    tokens, logprobs = [], []
    for i in range(case["rows"]):
        order = np.argsort(-x[i], kind="stable")
        k, t = int(v["top_k"][i]), float(v["temperature"][i])
        if t <= 0:
            tokens.append(order[0])
            logprobs.append(0.0)
            continue
        order = order[:k] if k > 0 else order
        y = (x[i][order] - x[i][order[0]]) / t
        w = np.exp(y)
        if v["top_p"][i] < 1:
            w = w[:1 + int(np.searchsorted(np.cumsum(w), float(v["top_p"][i]) * math.fsum(w)))]
        w = w[w >= v["min_p"][i]]  # weights fall along the order: what is left are its first ones
        by_index = np.argsort(order[:len(w)])
        c = np.cumsum(w[by_index])
        j = by_index[int(np.searchsorted(c, float(v["uniforms"][i]) * c[-1], side="right"))]
        tokens.append(order[j])
        logprobs.append(y[j] - math.log(math.fsum(w)))
    return {"tokens": np.array(tokens, np.int32), "logprobs": np.array(logprobs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "lora": _exact_lora, "sample": _exact_sample}[case["op"]](case, s)


# -------------------------------------------------------------------- work --


def work(case):
    """Bytes: every input once, every output once (of the pool the slots written).  Flops: the products and sums of the formulas."""
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 28), "flops": 3 * case["rows"] * case["vocab"]}
    n = _n_tokens(case)
    if case["op"] == "append":
        hq, hkv, d = (int(v) for v in case["heads"].split(","))
        outs = hq * (2 if case["rotated"] else 1) + 2 * hkv
        return {"bytes": n * (2 * d * (hq + 2 * hkv + outs) + 8), "flops": n * d * (hq + hkv) * 8}
    seqs, r, wi, wo = case["decodes"] + case["chunks"], case["rank"], case["width_in"], case["width_out"]
    with_adapter = n * (seqs - case["bare"]) / seqs
    used = min(case["adapters"], seqs - case["bare"])
    return {"bytes": 2 * (with_adapter * wi + 2 * n * wo + used * r * (wi + wo)), "flops": 2 * with_adapter * r * (wi + wo)}

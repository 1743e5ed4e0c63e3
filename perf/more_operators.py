"""Timed cases of three more operators of a ragged batch's serving step.

  append8  position rotation and the append of keys and values to a blocked KV pool of 8-bit
           codes with a scale for each (block, K or V, head) (``ds_kv8_rotary_append``)
  attend8  causal attention of every new token over its sequence's history in that pool
           (``ds_kv8_blocked_attention``)
  adjust   the rules of each request applied to its logits row before a token is drawn: biases of
           chosen tokens, penalties for repeated ones, a grammar's mask (``ds_ragged_adjust_logits``)

``run`` computes them in elementary torch operations, or, with ``own`` set, through the calls that a
user of the package makes.  ``exact`` computes the same from the definitions in 64 bits.

Definitions.
  codes:   e4m3 numbers (largest 448); a code c of a tile (block, K or V, head) with scale s stands for s * c.
           Scales are powers of two from 2^-40 to 2^40.
  append8: a key of a packed token at position p turns by the angle fp32(fp32(p) * fp32(theta^(-2k/d))) of
           each rotary pair.  A tile that gets tokens takes the smallest scale with which its new tokens'
           largest magnitude is at most 448 codes; if it holds earlier tokens of the sequence, at least the
           scale that it has, and where the scale grows their codes are rounded anew to it.  New
           elements are x / s, cut to +-448 and rounded to the nearest code (even in ties).
  attend8: out[t][h] = sum over u <= p of softmax_u(<rot(q_t,h), K_u> / sqrt(d)) V_u, with K and V the values of
           the codes and KV head floor(h / g).
  adjust:  z = x + the token's bias; where the token occurs in the request's history (prompt, then generated
           tokens) z / r if z > 0, else z * r; then z - f * c - p * [c > 0] with c its occurrences among the
           generated tokens; -inf where the mask has no bit for the token.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 64
DEV = "cuda"
F8 = torch.float8_e4m3fn

# (query heads, KV heads, head_dim) of the workloads, and small ones
HEADS = [(32, 32, 128), (32, 8, 128), (64, 8, 128), (4, 2, 64), (16, 2, 128), (8, 4, 64)]


def listed():
    return [
        # one request generating alone: the call's latency
        dict(name="append8_1_token", op="append8", decodes=1, chunks=0, tokens=0, max_seen=4000, heads="32,8,128", dtype="bf16",
             style="half", theta=5.0e5),
        # a full decode-only batch with one KV head per query head
        dict(name="append8_256_decodes", op="append8", decodes=256, chunks=0, tokens=0, max_seen=2047, heads="32,32,128",
             dtype="bf16", style="half", theta=1.0e4),
        # a mixed batch: prompt chunks and decodes, adjacent pairs, small heads
        dict(name="append8_mixed_small_heads", op="append8", decodes=61, chunks=5, tokens=1234, max_seen=900, heads="8,4,64",
             dtype="fp16", style="interleaved", theta=1.0e4),
        # two long prompt chunks of a large grouped-query layer
        dict(name="append8_2x8192", op="append8", decodes=0, chunks=2, tokens=16384, max_seen=4096, heads="64,8,128",
             dtype="bf16", style="half", theta=5.0e5),
        # one request generating alone over a history of 4000 tokens
        dict(name="attend8_1_row", op="attend8", decodes=1, chunks=0, tokens=0, max_seen=4000, heads="32,8,128", dtype="bf16",
             style="half", theta=5.0e5),
        # a full decode-only batch: the pool's bytes decide
        dict(name="attend8_256_decodes", op="attend8", decodes=256, chunks=0, tokens=0, max_seen=2047, heads="32,32,128",
             dtype="bf16", style="half", theta=1.0e4),
        # prompt chunks beside decodes with small heads
        dict(name="attend8_mixed_small_heads", op="attend8", decodes=61, chunks=5, tokens=1234, max_seen=900, heads="8,4,64",
             dtype="fp16", style="interleaved", theta=1.0e4),
        # two long prompt chunks of a large grouped-query layer: the matrix products decide
        dict(name="attend8_2x8192", op="attend8", decodes=0, chunks=2, tokens=16384, max_seen=4096, heads="64,8,128",
             dtype="bf16", style="half", theta=5.0e5),
        # one request with all its rules: latency
        dict(name="adjust_1_row", op="adjust", rows=1, vocab=32000, dtype="fp32", history=500, biased=16, masked=1.0),
        # a batch of requests with penalties and biases, a third of them under a grammar
        dict(name="adjust_256_mixed", op="adjust", rows=256, vocab=131072, dtype="bf16", history=4000, biased=32, masked=0.33),
        # an odd vocabulary (rows that start anywhere), every row under a grammar
        dict(name="adjust_64_masked", op="adjust", rows=64, vocab=50001, dtype="fp16", history=900, biased=0, masked=1.0),
        # long histories, 32-bit logits, penalties alone
        dict(name="adjust_256_long_histories", op="adjust", rows=256, vocab=131072, dtype="fp32", history=16000, biased=0,
             masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append8", "attend8", "adjust"])
    if op == "adjust":
        return dict(op=op, rows=_log_int(rng, 1, 256), vocab=_log_int(rng, 500, 131072), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    history=_log_int(rng, 1, 16000), biased=rng.choice([0, 1, 16, 200]), masked=rng.choice([0.0, 0.33, 1.0]))
    kind = rng.choice(["decode", "prompt", "mixed"])
    return dict(op=op, decodes=0 if kind == "prompt" else _log_int(rng, 1, 256), chunks=0 if kind == "decode" else _log_int(rng, 1, 12),
                tokens=0 if kind == "decode" else _log_int(rng, 32, 7900), max_seen=_log_int(rng, 1, 2047),
                heads="%d,%d,%d" % rng.choice(HEADS), dtype=rng.choice(["bf16", "fp16"]), style=rng.choice(["half", "interleaved"]),
                theta=rng.choice([1.0e4, 5.0e5, 1.0e6]))


def _heads(case):
    return tuple(int(v) for v in case["heads"].split(","))


def _batch(case):
    """(seen, new) of the batch's sequences, by the case alone: histories spread evenly up to max_seen, the longest for the
    first decode; from three chunks on they are of uneven lengths."""
    k, c, top = case["decodes"], case["chunks"], case["max_seen"]
    seen = [top * (k - i) // k for i in range(k)] + [top * (i + 1) // (2 * c) for i in range(c)]
    spare = case["tokens"] - 2 * c
    cuts = [0] + [spare * (4 * i + (i % 3 if c > 2 else 0)) // (4 * c) for i in range(1, c)] + [spare]
    return np.array(seen, np.int64), np.array([1] * k + [2 + cuts[i + 1] - cuts[i] for i in range(c)], np.int64)


def _lengths(case):
    """Tokens of each row's history, by the case alone."""
    return [case["history"] * (i + 1) // case["rows"] for i in range(case["rows"])]


def _on(a, dtype=torch.int64):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device=DEV)


def _power(e):
    """2^e for whole e."""
    return torch.bitwise_left_shift(e.int() + 127, 23).view(torch.float32)


def _scale_for(top):
    """The smallest power of two s from 2^-40 to 2^40 with top <= 448 s."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)  # 448 = 0.875 * 2^9
    return _power(torch.where(top > 0, e, -40).clamp(-40, 40))


# ------------------------------------------------------------------ inputs --


def _prepare_batch(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    hq, hkv, d = _heads(case)
    dt = DTYPES[case["dtype"]]
    seen, new = _batch(case)
    order = rs.permutation(len(new))
    seen, new = seen[order], new[order]
    total = seen + new
    need = (total + BLOCK - 1) // BLOCK
    blocks = int(need.sum()) + 3
    ids = rs.permutation(blocks).astype(np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    first = np.concatenate([[0], np.cumsum(new)])
    seq = np.repeat(np.arange(len(new)), new)
    pos = seen[seq] + np.arange(len(seq)) - first[seq]
    n, positions = len(seq), int(total.max())
    s = dict(case=case, hq=hq, hkv=hkv, d=d, n=n, seen=seen, new=new, first=first, need=need, ids=ids, at=at)
    s["qkv"] = torch.randn((n, (hq + 2 * hkv) * d), generator=gen, device=DEV).to(dt)
    # the cache: tiles as an append of normal values leaves them, of several magnitudes
    few = min(blocks, 256)
    x = torch.randn((few, 2, hkv, BLOCK, d), generator=gen, device=DEV)
    scale = _scale_for(x.abs().amax((3, 4)))
    codes = (x / scale[..., None, None]).to(F8).view(torch.uint8)
    s["codes"] = codes.repeat(-(-blocks // few), 1, 1, 1, 1)[:blocks].contiguous()
    size = _power(torch.randint(-1, 2, (blocks, 2, hkv), generator=gen, device=DEV))
    s["scales"] = (scale.repeat(-(-blocks // few), 1, 1)[:blocks] * size).contiguous()
    # the packed tokens: their tile rows, and the tiles that get tokens
    unit_key = at[seq] + pos // BLOCK
    units, unit = np.unique(unit_key, return_inverse=True)
    last_of = np.searchsorted(at, units, side="right") - 1
    older = np.clip(seen[last_of] - (units - at[last_of]) * BLOCK, 0, BLOCK)
    s["block"], s["slot"], s["pos"] = _on(ids[unit_key]), _on(pos % BLOCK), _on(pos)
    s["unit"], s["unit_block"], s["older"] = _on(unit), _on(ids[units]), _on(older)
    k = torch.arange(d // 2, device=DEV, dtype=torch.float64)
    s["freq"] = torch.pow(torch.tensor(np.float32(case["theta"]), dtype=torch.float64, device=DEV), -2 * k / d).float()
    turn = torch.arange(positions, device=DEV, dtype=torch.float32)[:, None] * s["freq"]
    s["cos"], s["sin"] = torch.cos(turn.double()).float(), torch.sin(turn.double()).float()
    # the sequences: decode rows with their blocks side by side, and chunks
    rows = np.nonzero(new == 1)[0]
    width = int(need[rows].max()) if len(rows) else 0
    table = np.zeros((len(rows), width), np.int64)
    inside = np.arange(width)[None, :] < need[rows][:, None]
    table[inside] = ids[(at[rows][:, None] + np.arange(width)[None, :])[inside]]
    s["row_token"], s["row_table"], s["row_len"] = _on(first[rows]), _on(table), _on(total[rows])
    s["chunks"] = [(int(first[i]), int(new[i]), int(seen[i]), _on(ids[at[i]:at[i + 1]])) for i in np.nonzero(new > 1)[0]]
    s["out"] = torch.zeros((n, hq * d), dtype=dt, device=DEV)
    if own:
        from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
        style = R.DS_ROPE_HALF if case["style"] == "half" else R.DS_ROPE_INTERLEAVED
        params = R.make_params(hq, hkv, d, case["dtype"], case["theta"], style)
        s["stream"] = torch.cuda.current_stream()
        s["layer"] = R.RaggedLayer(params, len(new), n, int(need.sum()), positions, stream=s["stream"])
        s["layer"].build(R.SeqDescs(seen, new, [ids[at[i]:at[i + 1]] for i in range(len(new))]), blocks)
        s["pool"] = R.make_kv8_pool(s["codes"], s["scales"])
    return s


def _prepare_adjust(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows, vocab, top, nb = case["rows"], case["vocab"], case["history"], min(case["biased"], case["vocab"])
    s = dict(case=case, logits=(2.2 * torch.randn((rows, vocab), generator=gen, device=DEV)).to(DTYPES[case["dtype"]]))
    # common tokens come again and again
    s["history"] = (vocab * torch.rand((rows, top), generator=gen, device=DEV).double() ** 3).int()
    length = np.array(_lengths(case))[rs.permutation(rows)]
    s["length"], s["prompt"] = _on(length, torch.int32), _on(length * rs.uniform(0.1, 0.9, rows), torch.int32)
    s["repetition"] = _on(rs.uniform(1.0, 1.3, rows), torch.float32)
    s["frequency"], s["presence"] = _on(rs.uniform(0.0, 0.7, rows), torch.float32), _on(rs.uniform(0.0, 0.7, rows), torch.float32)
    s["bias_ids"] = s["bias"] = s["bias_len"] = s["mask"] = s["mask_row"] = None
    if nb:
        s["bias_ids"] = torch.argsort(torch.rand((rows, vocab), generator=gen, device=DEV), 1)[:, :nb].int().contiguous()
        s["bias"] = 8 * torch.rand((rows, nb), generator=gen, device=DEV) - 4
        s["bias_len"] = torch.full((rows,), nb, dtype=torch.int32, device=DEV)
    under = int(math.ceil(case["masked"] * rows))
    if under:
        words = (vocab + 31) // 32
        # a grammar allows a run of tokens and some of the others
        bits = torch.randint(-2**31, 2**31, (under, words), generator=gen, device=DEV)
        bits &= torch.randint(-2**31, 2**31, (under, words), generator=gen, device=DEV)
        begin = torch.randint(0, words, (under, 1), generator=gen, device=DEV)
        word = torch.arange(words, device=DEV)
        s["mask"] = torch.where((word >= begin) & (word < begin + 1 + words // 8), -1, bits).int()
        which = np.full(rows, -1, np.int32)
        which[rs.permutation(rows)[:under]] = rs.permutation(under)
        s["mask_row"] = _on(which, torch.int32)
    s["out"] = torch.zeros_like(s["logits"])
    if own:
        from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
        s["stream"] = torch.cuda.current_stream()
        s["layer"] = R.RaggedLayer(R.make_params(1, 1, 64), rows, rows, rows, 1, stream=s["stream"])
        s["layer"].build(R.SeqDescs([0] * rows, [1] * rows, [np.array([i], np.int32) for i in range(rows)]), rows)
        s["rules"] = R.make_logit_rules(s["history"], s["length"], s["prompt"], s["repetition"], s["frequency"], s["presence"],
                                        s["bias_ids"], s["bias"], s["bias_len"], s["mask"], s["mask_row"])
    return s


def prepare(case, seed):
    return _prepare_adjust(case, seed) if case["op"] == "adjust" else _prepare_batch(case, seed)


# -------------------------------------------------------------- plain forms --


def _turned(x, c, s, style):
    """x [n, heads, d], c and s [n, 1, d/2]: each pair of the pairing rotated."""
    half = x.shape[-1] // 2
    if style == "half":
        x0, x1 = x[..., :half], x[..., half:]
        return torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)


def _coded(x, scale):
    return (x / scale).clamp(-448, 448).to(F8).view(torch.uint8)


def _append8(s):
    n, hq, hkv, d = s["n"], s["hq"], s["hkv"], s["d"]
    x = s["qkv"].view(n, hq + 2 * hkv, d)[:, hq:].float()
    c, t = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
    kv = torch.stack([_turned(x[:, :hkv], c, t, s["case"]["style"]), x[:, hkv:]], 1)  # [n, 2, heads, d]
    units, older = len(s["unit_block"]), s["older"][:, None, None]
    top = torch.zeros((units, 2, hkv), device=DEV).index_reduce_(0, s["unit"], kv.abs().amax(-1), "amax")
    had = s["scales"][s["unit_block"]]
    scale = torch.maximum(_scale_for(top), torch.where(older > 0, had, torch.zeros_like(had)))
    tiles = s["codes"][s["unit_block"]]
    kept = torch.arange(BLOCK, device=DEV)[:, None] < older[..., None, None]
    again = _coded(tiles.view(F8).float() * had[..., None, None], scale[..., None, None])
    s["codes"][s["unit_block"]] = torch.where(kept, again, tiles)
    s["scales"][s["unit_block"]] = scale
    s["codes"][s["block"], :, :, s["slot"]] = _coded(kv, scale[s["unit"]][..., None])
    return {"codes": s["codes"].view(F8), "scales": s["scales"]}


def _values(s, blocks, which):
    """K (0) or V (1) of some blocks in 32 bits: [..., heads, 64, d]."""
    return s["codes"][blocks, which].view(F8).float() * s["scales"][blocks, which][..., None, None]


def _attend8(s):
    n, hq, hkv, d = s["n"], s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    q = s["qkv"].view(n, hq + 2 * hkv, d)[:, :hq].float()
    q = _turned(q, s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None], s["case"]["style"]) / math.sqrt(d)
    out = torch.empty((n, hq, d), device=DEV)
    if s["row_table"].numel():  # all decode rows at once, side by side up to the longest
        rows, width = s["row_table"].shape
        k = _values(s, s["row_table"], 0)
        x = torch.matmul(q[s["row_token"]].view(rows, 1, hkv, g, d), k.transpose(-1, -2))  # [rows, blocks, heads, g, 64]
        del k
        u = torch.arange(width * BLOCK, device=DEV).view(1, width, 1, 1, BLOCK)
        x = torch.where(u < s["row_len"].view(-1, 1, 1, 1, 1), x, -math.inf)
        w = torch.exp(x - x.amax((1, 4), keepdim=True))
        w = w / w.sum((1, 4), keepdim=True)
        out[s["row_token"]] = torch.matmul(w, _values(s, s["row_table"], 1)).sum(1).view(rows, hq, d)
    for t0, new, seen, blocks in s["chunks"]:  # a chunk's scores are large: one sequence after another
        keys = seen + new
        k, v = (_values(s, blocks, i).transpose(0, 1).reshape(hkv, 1, -1, d)[:, :, :keys] for i in (0, 1))
        x = torch.matmul(q[t0:t0 + new].view(new, hkv, g, d).permute(1, 2, 0, 3), k.transpose(-1, -2))
        x.masked_fill_(torch.arange(keys, device=DEV) > seen + torch.arange(new, device=DEV)[:, None], -math.inf)
        x = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
        out[t0:t0 + new] = (torch.matmul(x, v) / x.sum(-1, keepdim=True)).permute(2, 0, 1, 3).reshape(new, hq, d)
        del x
    return {"out": out.to(s["qkv"].dtype).view(n, hq * d)}


def _adjust(s):
    x, vocab = s["logits"].float(), s["logits"].shape[1]
    place = torch.arange(s["history"].shape[1], device=DEV)
    inside, made = place < s["length"][:, None], place >= s["prompt"][:, None]
    h = s["history"].long()
    seen = torch.zeros(x.shape, dtype=torch.int32, device=DEV).scatter_add_(1, h, inside.int())
    count = torch.zeros_like(seen).scatter_add_(1, h, (inside & made).int())
    if s["bias"] is not None:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    r = s["repetition"][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["mask"] is not None:
        token = torch.arange(vocab, device=DEV)
        allowed = (torch.bitwise_right_shift(s["mask"][:, token // 32], (token % 32).int()) & 1) > 0
        x = torch.where(allowed[s["mask_row"].long().clamp(min=0)] | (s["mask_row"] < 0)[:, None], x, -math.inf)
    return {"logits": x.to(s["logits"].dtype)}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"append8": _append8, "attend8": _attend8, "adjust": _adjust}[op](s)
    from ragged_blocked_kv_raggedbatch_gb300 import ds_ragged as R
    if op == "append8":
        s["layer"].append8(s["qkv"], s["pool"])
        return {"codes": s["codes"].view(F8), "scales": s["scales"]}
    if op == "attend8":
        s["layer"].attention8(s["qkv"], s["pool"], s["out"])
        return {"out": s["out"]}
    R.ds_ragged_adjust_logits(s["layer"].meta, s["logits"], s["rules"], s["out"], s["stream"])
    return {"logits": s["out"]}


# ------------------------------------------------------- 64-bit definitions --


def _exact_rotated(case, s, lo, hi):
    """Heads lo..hi of qkv, rotated by the angles' complex factors."""
    n, d = s["n"], s["d"]
    x = s["qkv"].double().view(n, -1, d)[:, lo:hi]
    turn = (s["pos"].float()[:, None] * s["freq"]).double()
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]
    half = case["style"] == "half"
    z = x.reshape(n, -1, 2, d // 2).transpose(-1, -2) if half else x.reshape(n, -1, d // 2, 2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    return (z.transpose(-1, -2) if half else z).reshape(n, -1, d)


def _exact_codes(x):
    """The nearest e4m3 numbers of |x| <= 448 (even in ties): steps of 2^(e-3), at least 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append8(case, s):
    hq, hkv, n = s["hq"], s["hkv"], s["n"]
    new = torch.stack([_exact_rotated(case, s, hq, hq + hkv), s["qkv"].double().view(n, -1, s["d"])[:, hq + hkv:]], 1)
    codes, scales = s["codes"].view(F8).double(), s["scales"].double()
    block = s["block"].cpu().numpy()
    for b, older in zip(s["unit_block"].tolist(), s["older"].tolist()):
        mine = torch.as_tensor(np.nonzero(block == b)[0], device=DEV)
        x = new[mine]  # [tokens, 2, heads, d]
        top = x.abs().amax((0, 3)) / 448
        scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -60)))).clamp(2.0 ** -40, 2.0 ** 40)
        if older:
            scale = torch.maximum(scale, scales[b])
            codes[b, :, :, :older] = _exact_codes(codes[b, :, :, :older] * (scales[b] / scale)[..., None, None])
        codes[b][:, :, s["slot"][mine]] = _exact_codes((x / scale[..., None]).clamp(-448, 448)).permute(1, 2, 0, 3)
        scales[b] = scale
    return {"codes": codes, "scales": scales}


def _exact_attend8(case, s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    q = _exact_rotated(case, s, 0, hq)
    out = torch.empty_like(q)
    for i in range(len(s["new"])):
        t0, new, seen = int(s["first"][i]), int(s["new"][i]), int(s["seen"][i])
        blocks = _on(s["ids"][s["at"][i]:s["at"][i + 1]])
        hidden = torch.arange(seen + new, device=DEV) > seen + torch.arange(new, device=DEV)[:, None]
        step = hkv if new < 64 else 1
        for h in range(0, hkv, step):
            part = slice(h, h + step)
            kv = s["codes"][blocks][:, :, part].view(F8).double() * s["scales"][blocks][:, :, part].double()[..., None, None]
            kv = kv.permute(1, 2, 0, 3, 4).reshape(2, step, -1, d)[:, :, :seen + new]
            x = torch.einsum("thgd,hud->hgtu", q[t0:t0 + new].view(new, hkv, g, d)[:, part], kv[0]) * d ** -0.5
            w = torch.softmax(x.masked_fill_(hidden, -math.inf), -1)
            out[t0:t0 + new].view(new, hkv, g, d)[:, part] = torch.einsum("hgtu,hud->thgd", w, kv[1])
    return {"out": out.reshape(s["n"], hq * d)}


def _exact_adjust(case, s):
    x = s["logits"].double().cpu().numpy()
    v = {k: None if s[k] is None else s[k].cpu().numpy() for k in ("history", "length", "prompt", "repetition", "frequency", "presence",
                                                                   "bias_ids", "bias", "mask", "mask_row")}
    for i in range(case["rows"]):
        z, h = x[i], v["history"][i][:v["length"][i]]
        if v["bias"] is not None:
            z[v["bias_ids"][i]] += v["bias"][i]
        had = np.unique(h)
        z[had] = np.where(z[had] > 0, z[had] / float(v["repetition"][i]), z[had] * float(v["repetition"][i]))
        tokens, counts = np.unique(h[v["prompt"][i]:], return_counts=True)
        z[tokens] -= float(v["frequency"][i]) * counts + float(v["presence"][i])
        if v["mask"] is not None and v["mask_row"][i] >= 0:
            bits = np.unpackbits(v["mask"][v["mask_row"][i]].view(np.uint8), bitorder="little")[:case["vocab"]]
            z[bits == 0] = -np.inf
    return {"logits": x}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append8": _exact_append8, "attend8": _exact_attend8, "adjust": _exact_adjust}[case["op"]](case, s)


# -------------------------------------------------------------------- work --


def work(case):
    """Bytes: every input once, every output once (of the pool the tokens' own elements and their tiles' scales).  Flops: the
    products and sums of the formulas, a chunk's over the keys that each token sees."""
    if case["op"] == "adjust":
        rows, vocab, size = case["rows"], case["vocab"], 4 if case["dtype"] == "fp32" else 2
        mask = math.ceil(case["masked"] * rows) * ((vocab + 31) // 32) * 4
        return {"bytes": rows * (2 * vocab * size + 8 * min(case["biased"], vocab) + 28) + 4 * sum(_lengths(case)) + mask,
                "flops": 6 * sum(_lengths(case))}
    hq, hkv, d = _heads(case)
    seen, new = _batch(case)
    n, total = int(new.sum()), seen + new
    if case["op"] == "append8":
        tiles = int(((total - 1) // BLOCK - seen // BLOCK + 1).sum()) * 2 * hkv
        return {"bytes": n * (2 * hkv * d * 3 + 8) + 8 * tiles, "flops": n * hkv * d * 8}
    tiles = int(((total + BLOCK - 1) // BLOCK).sum()) * 2 * hkv
    pairs = int((new * seen + new * (new + 1) // 2).sum())
    return {"bytes": n * hq * d * 4 + int(total.sum()) * 2 * hkv * d + 4 * tiles, "flops": 4 * hq * d * pairs}

"""The key/value cache operators as a user's program calls them: rotary positions, appending new keys and values to a
paged cache with the rotation applied on the way, and the attention of a chunk of new tokens over that cache.

A case is a dict with "op" ("rope", "append" or "attend") and its sizes.  The sequences of a batch, their lengths and
so the work follow from the case alone; the values, the order of the pages and the positions follow from the seed.
"""
import math

import torch

#: False: `run` computes the operators in plain torch operations.  True: it calls this repository's operators.
own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BASE = 1000000.0  # base of the rotary frequencies


def listed():
    return [
        # the smallest call: one token's queries of the 27B-shaped layer (40 heads of 128), where latency counts
        {"name": "rope one token", "op": "rope", "tokens": 1, "heads": 40, "head_dim": 128, "rot_dim": 128,
         "interleaved": False, "far": 4096, "src": "f16", "dtype": "f16"},
        # queries of a long prompt, half of each head rotated in adjacent pairs, positions up to a million
        {"name": "rope prompt", "op": "rope", "tokens": 8191, "heads": 32, "head_dim": 128, "rot_dim": 64,
         "interleaved": True, "far": 1 << 20, "src": "bf16", "dtype": "bf16"},
        # one decode step of one sequence in the small dense model (32 query, 8 key/value heads): q, k, v as the
        # matrix-vector products leave them, in 32 bits
        {"name": "append one token", "op": "append", "seqs": 1, "new": 1, "context": 170, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "rot_dim": 128, "interleaved": False, "page": 16, "src": "f32", "dtype": "f16"},
        # prompts of several sequences that enter the cache together, ragged
        {"name": "append prompts", "op": "append", "seqs": 5, "new": 2048, "context": 4100, "ragged": True, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "rot_dim": 128, "interleaved": False, "page": 64, "src": "bf16", "dtype": "bf16"},
        # one decode step of one sequence, 27B-shaped layer, short context: latency
        {"name": "attend one token", "op": "attend", "seqs": 1, "new": 1, "context": 515, "ragged": False, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "window": 0, "page": 16, "dtype": "f16"},
        # one decode step of a served batch with ragged contexts
        {"name": "attend batch", "op": "attend", "seqs": 61, "new": 1, "context": 8192, "ragged": True, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "window": 0, "page": 64, "dtype": "f16"},
        # one decode step of one very long sequence
        {"name": "attend long context", "op": "attend", "seqs": 1, "new": 1, "context": 131067, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "window": 0, "page": 128, "dtype": "bf16"},
        # drafts of 16 tokens verified in 7 sequences, 27B-shaped layer
        {"name": "attend verify", "op": "attend", "seqs": 7, "new": 16, "context": 4001, "ragged": True, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "window": 0, "page": 32, "dtype": "f16"},
        # the 169-token prompt of the benchmark, 27B-shaped layer
        {"name": "attend prompt 169", "op": "attend", "seqs": 1, "new": 169, "context": 169, "ragged": False, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "window": 0, "page": 16, "dtype": "f16"},
        # chunks of ragged prompts in layers with a sliding window and heads of 64
        {"name": "attend window", "op": "attend", "seqs": 9, "new": 300, "context": 6001, "ragged": True, "heads": 32,
         "kv_heads": 4, "head_dim": 64, "window": 1024, "page": 24, "dtype": "bf16"},
        # a chunk of a long prompt that attends to what is in the cache already
        {"name": "attend chunk", "op": "attend", "seqs": 1, "new": 2048, "context": 16384, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "window": 0, "page": 128, "dtype": "bf16"},
        # a whole long prompt at once
        {"name": "attend prompt", "op": "attend", "seqs": 1, "new": 8192, "context": 8192, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "window": 0, "page": 64, "dtype": "f16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_any(rng):
    head_dim = rng.choice([64, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 10, 40])
    group = rng.choice([1, 4, 5, 8]) if kv_heads <= 8 else 1
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    case = {"op": op, "heads": kv_heads * group, "head_dim": head_dim, "dtype": rng.choice(["f16", "bf16"])}
    if op == "rope":
        case.update(tokens=_log_int(rng, 1, 8191), far=_log_int(rng, 4096, 1 << 20), src=rng.choice(["f32", case["dtype"]]),
                    rot_dim=rng.choice([head_dim, head_dim // 2]), interleaved=rng.random() < 0.5)
        return case
    case.update(kv_heads=kv_heads, seqs=_log_int(rng, 1, 96), page=rng.choice([16, 24, 32, 64, 128]),
                ragged=rng.random() < 0.7)
    new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
    case.update(new=new, context=new + _log_int(rng, 1, 32768) - 1)
    if op == "append":
        case.update(src=rng.choice(["f32", case["dtype"]]), rot_dim=rng.choice([head_dim, head_dim // 2]),
                    interleaved=rng.random() < 0.5)
    else:
        case.update(window=rng.choice([0, 0, 0, 128, 1000, 4096]))
    return case


def draw(rng):
    while True:
        case = _draw_any(rng)
        w = work(case)
        if w["flops"] > 5e11 or w["bytes"] > 6e8:
            continue
        if case["op"] != "rope":
            # the cache itself, and the plain form's score matrix, stay well below the largest listed case's
            if case["seqs"] * case["context"] * case["kv_heads"] * case["head_dim"] > 1 << 29:
                continue
            if case["op"] == "attend" and case["seqs"] * case["new"] * case["context"] * case["heads"] > 1 << 31:
                continue
        return case


def lengths(case):
    """(new tokens, context length with them) of each sequence: the case's, or, ragged, from an eighth of them up."""
    new, ctx = [], []
    for b in range(case["seqs"]):
        f = 1.0 if not case["ragged"] else 0.125 + 0.875 * ((0.37 + b * 0.6180339887498949) % 1.0)
        n = max(1, int(case["new"] * f))
        new.append(n)
        ctx.append(max(n, int(case["context"] * f)))
    return new, ctx


def _visible(n, c, window):
    """Query-key pairs of a sequence with n new tokens in a context of c."""
    return sum(min(p + 1, window) if window else p + 1 for p in range(c - n, c))


def work(case):
    s = BYTES[case["dtype"]]
    d = case["head_dim"]
    if case["op"] == "rope":
        values = case["tokens"] * case["heads"] * d
        return {"bytes": values * (BYTES[case["src"]] + s) + 4 * case["tokens"] + 4 * case["rot_dim"],
                "flops": 3 * case["tokens"] * case["heads"] * case["rot_dim"]}
    new, ctx = lengths(case)
    tokens = sum(new)
    if case["op"] == "append":
        values = tokens * (case["heads"] + 2 * case["kv_heads"]) * d
        tables = 4 * (2 * case["seqs"] + 1 + sum(-(-c // case["page"]) - (c - n) // case["page"] for n, c in zip(new, ctx)))
        return {"bytes": values * (BYTES[case["src"]] + s) + tables + 4 * case["rot_dim"],
                "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["rot_dim"]}
    w = case["window"]
    keys = sum(min(c, n + w - 1) if w else c for n, c in zip(new, ctx))
    pairs = sum(_visible(n, c, w) for n, c in zip(new, ctx))
    return {"bytes": 2 * keys * case["kv_heads"] * d * s + 2 * tokens * case["heads"] * d * s + 4 * (keys // case["page"] + 2 * case["seqs"] + 1),
            "flops": 4 * pairs * case["heads"] * d}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, d, h = DTYPES[case["dtype"]], case["head_dim"], case["heads"]

    def normal(*shape, dtype=kind):
        return torch.randn(shape, device="cuda", generator=g, dtype=torch.float32).to(dtype)

    state = {"case": case}
    if case["op"] != "attend":
        # the frequencies of the rotary positions, in 64 bits: made once for a model
        i = torch.arange(case["rot_dim"] // 2, device="cuda", dtype=torch.float64)
        state["inv_freq"] = torch.exp(i * (-2.0 * math.log(BASE) / case["rot_dim"]))
    if case["op"] == "rope":
        # the queries are a strided part of the packed projections
        t = case["tokens"]
        packed = normal(t, (h + 16) * d, dtype=DTYPES[case["src"]])
        state["x"] = packed[:, : h * d].view(t, h, d)
        state["positions"] = torch.randint(0, case["far"], (t,), device="cuda", generator=g, dtype=torch.int32)
        return state
    hk, page = case["kv_heads"], case["page"]
    new, ctx = lengths(case)
    need = [-(-c // page) for c in ctx]
    pages = sum(need) + 3
    # every sequence's pages lie anywhere in the cache, a few pages of the cache are free
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros((case["seqs"], max(need)), dtype=torch.int32, device="cuda")
    first = torch.tensor([sum(need[:b]) for b in range(case["seqs"])], device="cuda")
    held = torch.arange(max(need), device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[held] = order[(first[:, None] + torch.arange(max(need), device="cuda")[None, :])[held]]
    state["block_table"] = table
    state["query_start"] = torch.tensor([sum(new[:b]) for b in range(case["seqs"] + 1)], dtype=torch.int32, device="cuda")
    state["context_lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    state["max_new"], state["max_context"] = max(new), max(ctx)
    tokens = sum(new)
    state["k_cache"] = normal(pages, hk, page, d)
    state["v_cache"] = normal(pages, hk, page, d)
    if case["op"] == "append":
        packed = normal(tokens, (h + 2 * hk) * d, dtype=DTYPES[case["src"]])
        state["q"] = packed[:, : h * d].view(tokens, h, d)
        state["k"] = packed[:, h * d : (h + hk) * d].view(tokens, hk, d)
        state["v"] = packed[:, (h + hk) * d :].view(tokens, hk, d)
    else:
        # queries somewhat aligned with some keys, so that the probabilities are not flat
        state["q"] = 2.0 * normal(tokens, h, d, dtype=torch.float32)
        state["q"] = state["q"].to(kind)
        state["scale"] = 1.0 / math.sqrt(d)
    if own:
        import q4_dequant_gemv_block_amd as q4
        state["cache"] = q4.KVCache(state["k_cache"], state["v_cache"])
        state["batch"] = q4.KVBatch(state["block_table"], state["query_start"], state["context_lens"],
                                    max_query_len=state["max_new"], max_context_len=state["max_context"])
    return state


def run(state):
    case = state["case"]
    if own:
        import q4_dequant_gemv_block_amd as q4
        layout = "interleaved" if case.get("interleaved") else "half"
        if case["op"] == "rope":
            out = torch.empty(state["x"].shape, dtype=DTYPES[case["dtype"]], device="cuda")
            return q4.q4_rope(state["x"], state["positions"], state["inv_freq"], layout=layout, out=out)
        if case["op"] == "append":
            q = q4.q4_kv_append(state["cache"], state["batch"], state["k"], state["v"], q=state["q"],
                                inv_freq=state["inv_freq"], layout=layout)
            return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        return q4.q4_attention_paged(state["cache"], state["batch"], state["q"], scale=state["scale"], window=case["window"])
    if case["op"] == "rope":
        return _rotate(state["x"], state["positions"], state["inv_freq"], case["interleaved"]).to(DTYPES[case["dtype"]])
    if case["op"] == "append":
        return _append(state, case)
    return _attend(state, case)


def _rotate(x, positions, inv_freq, interleaved):
    """x (tokens, heads, dim) in 32 bits with its leading pairs turned by positions * inv_freq."""
    angle = positions.to(torch.float64)[:, None] * inv_freq
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    r = 2 * inv_freq.numel()
    x = x.float()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _places(state, tokens):
    """The sequence of each new token, its index among that sequence's new tokens and its position."""
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    start = state["query_start"]
    seq = torch.searchsorted(start, t, right=True) - 1
    index = t - start[seq]
    position = state["context_lens"][seq] - (start[seq + 1] - start[seq]) + index
    return seq, index.long(), position.long()


def _append(state, case):
    kind, page = DTYPES[case["dtype"]], case["page"]
    seq, _, position = _places(state, state["k"].shape[0])
    where = state["block_table"][seq, position // page].long(), position % page
    q = _rotate(state["q"], position, state["inv_freq"], case["interleaved"]).to(kind)
    k = _rotate(state["k"], position, state["inv_freq"], case["interleaved"]).to(kind)
    state["k_cache"][where[0], :, where[1]] = k
    state["v_cache"][where[0], :, where[1]] = state["v"].to(kind)
    return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}


def _attend(state, case):
    q, table = state["q"], state["block_table"].long()
    tokens, h, d = q.shape
    hk, seqs = case["kv_heads"], case["seqs"]
    group, most = h // hk, state["max_new"]
    # keys and values of every sequence, its pages one after the other: (sequences, kv heads, keys, dim)
    k = state["k_cache"][table].transpose(1, 2).flatten(2, 3).float()
    v = state["v_cache"][table].transpose(1, 2).flatten(2, 3).float()
    start, ctx = state["query_start"].long(), state["context_lens"].long()
    row = torch.arange(most, device="cuda")
    x = q[(start[:-1, None] + row).clamp(max=tokens - 1)].float()
    x = x.view(seqs, most, hk, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, hk, most * group, d)
    position = (ctx - (start[1:] - start[:-1]))[:, None] + row
    key = torch.arange(k.shape[2], device="cuda")
    seen = (key <= position[..., None]) & (key < ctx[:, None, None])
    if case["window"]:
        seen &= key > position[..., None] - case["window"]
    seen = seen[:, None, :, None, :]
    s = torch.matmul(x, k.transpose(-1, -2).contiguous()).mul_(state["scale"]).view(seqs, hk, most, group, -1)
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hk, most * group, -1), v).view(seqs, hk, most, group, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    seq, index, _ = _places(state, tokens)
    return o.permute(0, 2, 1, 3, 4)[seq, index].reshape(tokens, h, d).to(q.dtype)


def exact(case, seed):
    """What `run` returns, in 64 bits, one sequence and head after the other."""
    state = prepare(case, seed)
    if case["op"] == "rope":
        return _turn_exact(state["x"], state["positions"].double(), case)
    new, ctx = lengths(case)
    page, d = case["page"], case["head_dim"]
    first = [sum(new[:b]) for b in range(case["seqs"] + 1)]
    if case["op"] == "append":
        at = torch.cat([torch.arange(c - n, c, device="cuda") for n, c in zip(new, ctx)])
        q, k = _turn_exact(state["q"], at.double(), case), _turn_exact(state["k"], at.double(), case)
        caches = state["k_cache"].double(), state["v_cache"].double()
        for b in range(case["seqs"]):
            part = slice(first[b], first[b + 1])
            pos = at[part]
            slot = state["block_table"][b].long().index_select(0, pos // page) * page + pos % page
            for cache, rows in zip(caches, (k[part], state["v"][part].double())):
                flat = cache.permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], d)
                flat.index_copy_(0, slot, rows)
                cache.copy_(flat.view(-1, page, case["kv_heads"], d).permute(0, 2, 1, 3))
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        n, c = new[b], ctx[b]
        low = max(0, c - n - case["window"] + 1) if case["window"] else 0
        pos = torch.arange(low, c, device="cuda")
        pages = state["block_table"][b].long()[pos // page]
        for hk in range(case["kv_heads"]):
            k = state["k_cache"][pages, hk, pos % page].double()
            v = state["v_cache"][pages, hk, pos % page].double()
            step = max(1, (1 << 27) // max(1, group * (c - low)))
            for i in range(0, n, step):
                rows = torch.arange(i, min(n, i + step), device="cuda")
                x = state["q"][first[b] + rows, hk * group : (hk + 1) * group].double()
                s = torch.einsum("tgd,kd->tgk", x, k) * state["scale"]
                gone = pos[None, :] > (c - n + rows)[:, None]
                if case["window"]:
                    gone |= pos[None, :] <= (c - n + rows)[:, None] - case["window"]
                p = torch.softmax(s.masked_fill(gone[:, None, :], -math.inf), -1)
                out[first[b] + rows, hk * group : (hk + 1) * group] = torch.einsum("tgk,kd->tgd", p, v)
    return out


def _turn_exact(x, position, case):
    """The pairs as complex numbers, multiplied by exp(i * angle)."""
    half = case["rot_dim"] // 2
    x = x.double()
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    angle = position[:, None] * torch.exp(i * (-2.0 * math.log(BASE) / case["rot_dim"]))
    unit = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    out = x.clone()
    if case["interleaved"]:
        z = torch.complex(x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]) * unit
        out[..., 0 : 2 * half : 2], out[..., 1 : 2 * half : 2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :half], x[..., half : 2 * half]) * unit
        out[..., :half], out[..., half : 2 * half] = z.real, z.imag
    return out

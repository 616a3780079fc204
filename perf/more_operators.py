"""One step of greedy decoding with trees of drafted tokens, operator by operator, as a user's program calls them: the
step's block tables, slots and masks from request lengths, per-head norms of queries and keys with the rotation on the
way into the cache, attention of the drafted tree over the cache, penalties, biases and grammars on the logits with the
greedy pick, and the path taken with the cache's slots closed up behind it.

A case is a dict with "op" ("assign", "norm", "append", "tree", "logits" or "settle") and its sizes.  The sequences of
a batch and their lengths follow from the case alone; the values, the trees and the order of the pages follow from the
seed.
"""
import math

import torch

#: False: `run` computes the operators in plain torch operations.  True: it calls this repository's operators.
own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BASE = 1000000.0  # base of the rotary frequencies
EPS = 1e-6
VOCAB = 151936


def listed():
    return [
        # the tables of a decode step of a small batch: the smallest call, where latency counts
        {"name": "assign decode", "op": "assign", "seqs": 8, "new": 1, "past": 2048, "ragged": True, "page": 16, "tree": False},
        # drafted trees of a large served batch over long block tables: positions by depth, slots, ancestors' masks
        {"name": "assign trees", "op": "assign", "seqs": 256, "new": 64, "past": 16384, "ragged": True, "page": 16, "tree": True},
        # a decode step of one sequence in the small dense model (32 query, 8 key/value heads), products in 32 bits
        {"name": "append one token", "op": "append", "seqs": 1, "new": 1, "past": 170, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "rot_dim": 128, "interleaved": False, "page": 16, "src": "f32", "dtype": "f16"},
        # ragged prompts that enter the cache together
        {"name": "append prompts", "op": "append", "seqs": 5, "new": 2048, "past": 2052, "ragged": True, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "rot_dim": 128, "interleaved": False, "page": 64, "src": "bf16", "dtype": "bf16"},
        # a tree of 16 drafted tokens of one sequence, 27B-shaped layer, short context
        {"name": "tree one sequence", "op": "tree", "seqs": 1, "new": 16, "past": 515, "ragged": False, "heads": 40,
         "kv_heads": 40, "head_dim": 128, "window": 0, "page": 16, "dtype": "f16"},
        # trees of up to 33 tokens in a served batch with ragged contexts
        {"name": "tree batch", "op": "tree", "seqs": 16, "new": 33, "past": 6001, "ragged": True, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "window": 0, "page": 64, "dtype": "bf16"},
        # wide trees over long contexts
        {"name": "tree long context", "op": "tree", "seqs": 3, "new": 64, "past": 32768, "ragged": False, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "window": 0, "page": 128, "dtype": "f16"},
        # the greedy pick of one sequence with penalties and a grammar, vocabulary of the benchmark
        {"name": "logits one row", "op": "logits", "seqs": 1, "new": 1, "past": 600, "ragged": False, "vocab": VOCAB,
         "biases": 0, "grammar": True, "tree": False, "out": False, "dtype": "f32"},
        # the nodes of drafted trees: each sees its ancestors' tokens beside its sequence's
        {"name": "logits trees", "op": "logits", "seqs": 4, "new": 16, "past": 3000, "ragged": True, "vocab": VOCAB,
         "biases": 40, "grammar": True, "tree": True, "out": False, "dtype": "f32"},
        # a decode step of a large batch whose logits go on to sampling
        {"name": "logits batch", "op": "logits", "seqs": 192, "new": 1, "past": 4096, "ragged": True, "vocab": VOCAB,
         "biases": 300, "grammar": False, "tree": False, "out": True, "dtype": "f32"},
        # the path through one sequence's tree, one layer's cache
        {"name": "settle one sequence", "op": "settle", "seqs": 1, "new": 16, "past": 170, "ragged": False, "layers": 1,
         "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "f16"},
        # a served batch, the caches of 36 layers
        {"name": "settle batch", "op": "settle", "seqs": 48, "new": 48, "past": 140, "ragged": True, "layers": 36,
         "kv_heads": 8, "head_dim": 128, "page": 16, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_any(rng):
    op = rng.choice(["assign", "norm", "append", "tree", "tree", "logits", "logits", "settle"])
    head_dim = rng.choice([64, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 10, 40])
    group = rng.choice([1, 4, 5, 8]) if kv_heads <= 8 else 1
    case = {"op": op, "ragged": rng.random() < 0.7, "seqs": _log_int(rng, 1, 300 if op == "assign" else 96),
            "page": rng.choice([16, 24, 32, 64, 128])}
    nodes = _log_int(rng, 2, 200)
    if op == "assign":
        case["tree"] = rng.random() < 0.6
        case["new"] = nodes if case["tree"] else 1 if rng.random() < 0.5 else _log_int(rng, 2, 3000)
        case["past"] = _log_int(rng, 1, 32768) - 1
        return case
    if op == "logits":
        case.update(tree=rng.random() < 0.5, vocab=_log_int(rng, 1000, 260000), past=_log_int(rng, 1, 20000),
                    biases=rng.choice([0, 0, 7, 300]), grammar=rng.random() < 0.5, out=rng.random() < 0.5,
                    dtype=rng.choice(["f32", "f32", "f16", "bf16"]))
        case["new"] = min(nodes, 64) if case["tree"] else 1
        del case["page"]
        return case
    case.update(head_dim=head_dim, dtype=rng.choice(["f16", "bf16"]))
    if op == "settle":
        case.update(kv_heads=kv_heads, layers=_log_int(rng, 1, 40), new=nodes, past=_log_int(rng, 1, 500) - 1)
        return case
    case.update(heads=kv_heads * group, kv_heads=kv_heads)
    if op == "tree":
        case.update(new=nodes, past=_log_int(rng, 1, 32768) - 1, window=rng.choice([0, 0, 0, 128, 1000, 4096]))
        return case
    case.update(rot_dim=rng.choice([head_dim, head_dim // 2]), interleaved=rng.random() < 0.5,
                src=rng.choice(["f32", case["dtype"]]), new=1 if rng.random() < 0.4 else _log_int(rng, 2, 4096))
    case["past"] = _log_int(rng, 1, 8192) - 1
    return case


def draw(rng):
    while True:
        case = _draw_any(rng)
        w = work(case)
        if w["bytes"] > 5e8 or w["flops"] > 1.6e11:
            continue
        if "kv_heads" in case:
            # the cache itself stays below the largest listed case's
            held = case["seqs"] * (case["past"] + case["new"] + case["page"]) * case["kv_heads"] * case["head_dim"] * case.get("layers", 1)
            if held > 1 << 28:
                continue
        if case["op"] == "tree" and case["seqs"] * case["new"] * (case["past"] + case["new"]) * case["heads"] > 1 << 28:
            continue
        if case["op"] == "logits" and case["seqs"] * case["new"] * case["vocab"] > 192 * VOCAB:
            continue
        return case


def lengths(case):
    """(new tokens, tokens before them) of each sequence: the case's, or, ragged, from an eighth of them up."""
    new, past = [], []
    for b in range(case["seqs"]):
        f = 1.0 if not case["ragged"] else 0.125 + 0.875 * ((0.37 + b * 0.6180339887498949) % 1.0)
        new.append(max(1, int(case["new"] * f)))
        past.append(int(case["past"] * f))
    return new, past


def work(case):
    new, past = lengths(case)
    tokens, seqs = sum(new), case["seqs"]
    op = case["op"]
    if op == "assign":
        columns = _columns(case)
        each = 12 + (4 + 8 * _words(case) if case["tree"] else 0)
        return {"bytes": 8 * seqs * columns + 28 * seqs + each * tokens, "flops": tokens}
    if op == "logits":
        values = tokens * case["vocab"]
        lists = 4 * sum(past) + 8 * seqs * case["biases"] + (4 + 8 * _words(case)) * tokens * case["tree"]
        return {"bytes": values * (BYTES[case["dtype"]] + 4 * case["out"]) + values // 8 * case["grammar"] + lists + 4 * tokens,
                "flops": 4 * values}
    d, s = case["head_dim"], BYTES[case["dtype"]]
    if op == "settle":
        # about a third of a tree's depth is taken, and all of that but the root changes its slot
        kept = sum(max(0, min(4, n - 1)) for n in new)
        return {"bytes": 4 * kept * case["layers"] * case["kv_heads"] * d * s + 16 * tokens, "flops": tokens}
    if op in ("norm", "append"):
        heads = case["heads"] + (2 * case["kv_heads"] if op == "append" else 0)
        turned = case["heads"] + (case["kv_heads"] if op == "append" else 0)
        return {"bytes": tokens * heads * d * (BYTES[case["src"]] + s) + 8 * tokens + 4 * case["rot_dim"] + 8 * d,
                "flops": tokens * turned * (4 * d + 3 * case["rot_dim"])}
    w = case["window"]
    keys = sum(n + (min(p, w) if w else p) for n, p in zip(new, past))
    pairs = sum(n * (min(p, w) if w else p) + 6 * n for n, p in zip(new, past))
    return {"bytes": 2 * keys * case["kv_heads"] * d * s + 2 * tokens * case["heads"] * d * s + 8 * _words(case) * tokens + 4 * (keys // case["page"] + 2 * seqs + 1),
            "flops": 4 * pairs * case["heads"] * d}


def _words(case):
    """64-bit words of a token's mask."""
    return -(-case["new"] // 64)


def _columns(case):
    """Pages a row of the block table holds."""
    return -(-(case["past"] + case["new"]) // case["page"]) + 1


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _places(start, tokens):
    """The sequence of each new token and its index among that sequence's new tokens."""
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(start, t, right=True) - 1
    return seq, (t - start[seq]).long()


def _grow(index, g):
    """A parent for every token that is not its sequence's first, more often a late one; -1 for the first."""
    u = torch.rand(index.shape, device="cuda", generator=g, dtype=torch.float64).sqrt()
    return torch.where(index > 0, (u * index).long().clamp(max=index - 1), index.new_tensor(-1)).to(torch.int32)


def _ancestors(parents, start, most):
    """[sequences, most, most] of truth values: whether a new token is another's ancestor, or itself."""
    tokens = parents.shape[0]
    seq, index = _places(start, tokens)
    step = torch.zeros((start.shape[0] - 1, most, most), dtype=torch.float64, device="cuda")
    has = parents >= 0
    step[seq[has], index[has], parents[has].long()] = 1.0
    step += torch.eye(most, dtype=torch.float64, device="cuda")
    return torch.linalg.matrix_power(step, most) > 0


def _mask_words(closure, start, tokens, words):
    """The rows of `closure` as bits of 64-bit words [tokens, words]."""
    seq, index = _places(start, tokens)
    rows = closure[seq, index]
    rows = torch.nn.functional.pad(rows, (0, 64 * words - rows.shape[1])).view(tokens, words, 64)
    return (rows.long() << torch.arange(64, device="cuda")).sum(-1)


def _bits(mask, start, most):
    """[sequences, most, 64 words] of truth values from the masks of the new tokens."""
    tokens, words = mask.shape
    seq, index = _places(start, tokens)
    rows = ((mask[:, :, None] >> torch.arange(64, device="cuda")) & 1).bool().view(tokens, 64 * words)
    out = torch.zeros((start.shape[0] - 1, most, 64 * words), dtype=torch.bool, device="cuda")
    out[seq, index] = rows
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, seqs = case["op"], case["seqs"]
    new, past = lengths(case)
    tokens = sum(new)
    state = {"case": case, "most": max(new), "tokens": tokens}
    state["query_start"] = _int32([sum(new[:b]) for b in range(seqs + 1)])
    state["past_lens"], state["new_lens"] = _int32(past), _int32(new)
    state["context_lens"] = state["past_lens"] + state["new_lens"]
    if op == "assign":
        _prepare_assign(state, g)
    elif op == "logits":
        _prepare_logits(state, g)
    else:
        _prepare_heads(state, g)
    return state


def _prepare_assign(state, g):
    """The last step's block table, in which each sequence holds the pages of the tokens it has, and the free pages."""
    case, seqs, columns = state["case"], state["case"]["seqs"], _columns(state["case"])
    held = -(-state["past_lens"] // case["page"])
    pages = seqs * columns + 5
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = order[: seqs * columns].view(seqs, columns).clone()
    has = torch.arange(columns, device="cuda", dtype=torch.int32) < held[:, None]
    state["free_pages"] = torch.cat((order[seqs * columns:], table[~has]))
    # enough for all but the last few sequences of a large batch
    state["free_count"] = _int32([state["free_pages"].shape[0]])
    need = (-(-state["context_lens"] // case["page"]) - held).sum()
    if seqs > 100:
        state["free_count"] = (need - 3).clamp(min=0).to(torch.int32).view(1)
    state["block_table"], state["held"] = table.masked_fill(~has, -1), held
    state["parents"] = None
    if case["tree"]:
        state["parents"] = _grow(_places(state["query_start"], state["tokens"])[1], g)
    if own:
        import q4_dequant_gemv_block_amd as q4
        state["step"] = q4.KVStep(seqs, columns, case["page"], state["tokens"], _words(case) if case["tree"] else 0)


def _prepare_logits(state, g):
    case, seqs, vocab = state["case"], state["case"]["seqs"], state["case"]["vocab"]
    tokens = state["tokens"]
    state["logits"] = (2.5 * torch.randn((tokens, vocab), device="cuda", generator=g)).to(DTYPES[case["dtype"]])
    # token numbers as a text has them: some far more often than others
    def text(*shape):
        u = torch.rand(shape, device="cuda", generator=g, dtype=torch.float64)
        return (u ** 4 * vocab).long().clamp(max=vocab - 1).to(torch.int32)

    state["history"] = text(seqs, case["past"] + 8)
    state["prompt_lens"] = state["past_lens"] // 3
    state["draft"] = text(tokens) if case["tree"] else None
    state["mask"] = None
    if case["tree"]:
        parents = _grow(_places(state["query_start"], tokens)[1], g)
        state["mask"] = _mask_words(_ancestors(parents, state["query_start"], state["most"]), state["query_start"], tokens, _words(case))

    def between(lo, hi):
        return lo + (hi - lo) * torch.rand((seqs,), device="cuda", generator=g)

    state["repetition"], state["presence"], state["frequency"] = between(1.0, 1.5), between(0.0, 1.0), between(0.0, 0.7)
    state["bias_start"] = state["bias_tokens"] = state["bias_values"] = None
    if case["biases"]:
        n = case["biases"]
        state["bias_start"] = _int32([n * b for b in range(seqs + 1)])
        first = torch.randint(0, vocab, (seqs, 1), device="cuda", generator=g)
        # n different tokens of each sequence
        state["bias_tokens"] = ((first + torch.arange(n, device="cuda") * (vocab // n)) % vocab).to(torch.int32).view(-1)
        state["bias_values"] = 3.0 * torch.randn((seqs * n,), device="cuda", generator=g)
    state["allowed"] = None
    if case["grammar"]:
        state["allowed"] = torch.randint(-(1 << 31), (1 << 31), (tokens, -(-vocab // 32)), device="cuda", generator=g).to(torch.int32)
    if own:
        import q4_dequant_gemv_block_amd as q4
        state["rules"] = q4.LogitRules(
            query_start=state["query_start"], history=state["history"], history_lens=state["past_lens"],
            prompt_lens=state["prompt_lens"], draft=state["draft"], mask=state["mask"], repetition=state["repetition"],
            presence=state["presence"], frequency=state["frequency"], bias_start=state["bias_start"],
            bias_tokens=state["bias_tokens"], bias_values=state["bias_values"], allowed=state["allowed"])


def _prepare_heads(state, g):
    case, op, seqs = state["case"], state["case"]["op"], state["case"]["seqs"]
    kind, d, page, tokens = DTYPES[case["dtype"]], case["head_dim"], case["page"], state["tokens"]

    def normal(*shape, dtype=kind):
        return torch.randn(shape, device="cuda", generator=g, dtype=torch.float32).to(dtype)

    if op in ("norm", "append"):
        # the frequencies of the rotary positions, in 64 bits, and the norms' gains: of the model
        i = torch.arange(case["rot_dim"] // 2, device="cuda", dtype=torch.float64)
        state["inv_freq"] = torch.exp(i * (-2.0 * math.log(BASE) / case["rot_dim"]))
        state["q_gain"], state["k_gain"] = (1.0 + 0.2 * normal(d, dtype=torch.float32)).to(kind), (1.0 + 0.2 * normal(d, dtype=torch.float32)).to(kind)
    if op == "norm":
        # the queries are a strided part of the packed projections
        h = case["heads"]
        state["x"] = normal(tokens, (h + 16) * d, dtype=DTYPES[case["src"]])[:, : h * d].view(tokens, h, d)
        state["positions"] = torch.randint(0, 1 << 20, (tokens,), device="cuda", generator=g, dtype=torch.int32)
        return
    hk, columns = case["kv_heads"], _columns(case)
    new, past = lengths(case)
    need = [-(-(n + p) // page) for n, p in zip(new, past)]
    pages = sum(need) + 3
    # every sequence's pages lie anywhere in the cache, a few pages of the cache are free
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros((seqs, columns), dtype=torch.int32, device="cuda")
    held = torch.arange(columns, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[held] = order[: sum(need)]
    state["block_table"] = table
    layers = case.get("layers", 1)
    state["k_cache"], state["v_cache"] = normal(layers, pages, hk, page, d), normal(layers, pages, hk, page, d)
    if op == "append":
        h = case["heads"]
        packed = normal(tokens, (h + 2 * hk) * d, dtype=DTYPES[case["src"]])
        state["q"] = packed[:, : h * d].view(tokens, h, d)
        state["k"] = packed[:, h * d : (h + hk) * d].view(tokens, hk, d)
        state["v"] = packed[:, (h + hk) * d :].view(tokens, hk, d)
    else:
        state["parents"] = _grow(_places(state["query_start"], tokens)[1], g)
    if op == "tree":
        # queries somewhat aligned with some keys, so that the probabilities are not flat
        state["q"] = (2.0 * normal(tokens, case["heads"], d, dtype=torch.float32)).to(kind)
        state["scale"] = 1.0 / math.sqrt(d)
        state["mask"] = _mask_words(_ancestors(state["parents"], state["query_start"], state["most"]), state["query_start"], tokens, _words(case))
    if op == "settle":
        # the trunk's choice behind every node, and drafts of which about two thirds are what it chose
        state["choice"] = torch.randint(0, VOCAB, (tokens,), device="cuda", generator=g, dtype=torch.int32)
        seq, index = _places(state["query_start"], tokens)
        other = torch.randint(0, VOCAB, (tokens,), device="cuda", generator=g, dtype=torch.int32)
        parent_row = (state["query_start"][seq] + state["parents"].clamp(min=0)).long()
        right = (torch.rand((tokens,), device="cuda", generator=g) < 0.65) & (index > 0)
        state["draft"] = torch.where(right, state["choice"][parent_row], other)
        state["history"] = torch.zeros((seqs, case["past"] + case["new"]), dtype=torch.int32, device="cuda")
    if own:
        import q4_dequant_gemv_block_amd as q4
        caches = [q4.KVCache(state["k_cache"][i], state["v_cache"][i]) for i in range(layers)]
        state["cache"] = caches[0] if op != "settle" else q4.KVLayers(caches)
        state["batch"] = q4.KVBatch(table, state["query_start"], state["context_lens"], max_query_len=max(new),
                                    max_context_len=max(n + p for n, p in zip(new, past)))


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import q4_dequant_gemv_block_amd as q4
        layout = "interleaved" if case.get("interleaved") else "half"
        if op == "assign":
            step = q4.q4_kv_assign(state["step"], state["block_table"], state["held"], state["past_lens"], state["new_lens"],
                                   state["free_pages"], state["free_count"], parents=state["parents"])
            return {"block_table": step.block_table, "held": step.held, "query_start": step.query_start,
                    "context_lens": step.context_lens, "missing": step.missing, "free_count": step.free_count,
                    "positions": step.positions, "slots": step.slots, "mask": step.mask}
        if op == "norm":
            out = torch.empty(state["x"].shape, dtype=DTYPES[case["dtype"]], device="cuda")
            return q4.q4_norm_rope(state["x"], state["q_gain"], eps=EPS, positions=state["positions"], inv_freq=state["inv_freq"],
                                   layout=layout, out=out)
        if op == "append":
            q = q4.q4_kv_append_norm(state["cache"], state["batch"], state["k"], state["v"], q=state["q"], k_gain=state["k_gain"],
                                     q_gain=state["q_gain"], eps=EPS, inv_freq=state["inv_freq"], layout=layout)
            return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
        if op == "tree":
            return q4.q4_attention_tree(state["cache"], state["batch"], state["q"], state["mask"], scale=state["scale"], window=case["window"])
        if op == "logits":
            out = torch.empty(state["logits"].shape, dtype=torch.float32, device="cuda") if case["out"] else None
            return {"tokens": q4.q4_logits_argmax(state["logits"], state["rules"], out=out), "logits": out}
        accepted, tokens, path, lens = q4.q4_tree_accept(state["batch"], state["choice"], state["draft"], parents=state["parents"],
                                                         history=state["history"])
        q4.q4_kv_move(state["cache"], state["batch"], path, accepted)
        return {"accepted": accepted, "tokens": tokens, "path": path, "lens": lens, "history": state["history"],
                "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    if op == "assign":
        return _assign(state, case)
    if op == "norm":
        x = _normed(state["x"], state["q_gain"])
        return _rotate(x, state["positions"], state["inv_freq"], case["interleaved"]).to(DTYPES[case["dtype"]])
    if op == "append":
        return _append(state, case)
    if op == "tree":
        return _attend(state, case)
    if op == "logits":
        return _pick(state, case)
    return _settle(state, case)


def _assign(state, case):
    past, new, held, table = state["past_lens"], state["new_lens"], state["held"], state["block_table"]
    page, seqs = case["page"], case["seqs"]
    context = past + new
    start = torch.nn.functional.pad(torch.cumsum(new, 0, dtype=torch.int32), (1, 0))
    lack = (-(-context // page) - held).clamp(min=0)
    upto = torch.cumsum(lack, 0, dtype=torch.int32)
    count = state["free_count"]
    served = (upto <= count) | (lack == 0)
    taken = torch.where(served, lack, 0)
    # column c of a served sequence that it did not hold: the free list from its end, in the order of sequences
    column = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)
    nth = (upto - lack)[:, None] + column - held[:, None]
    fresh = served[:, None] & (column >= held[:, None]) & (column < (held + lack)[:, None])
    free = state["free_pages"][(count - 1 - nth).clamp(min=0, max=state["free_pages"].shape[0] - 1)]
    table = torch.where(fresh, free, table)
    tokens = state["tokens"]
    seq, index = _places(start, tokens)
    place = past[seq].long() + index
    of = table[seq, place // page].long()
    slots = torch.where(of >= 0, of * page + place % page, -1)
    positions, mask = place, []
    if state["parents"] is not None:
        closure = _ancestors(state["parents"], start, state["most"])
        positions = past[seq].long() + closure[seq, index].sum(-1) - 1
        mask = _mask_words(closure, start, tokens, _words(case))
    return {"block_table": table, "held": held + taken, "query_start": start, "context_lens": context,
            "missing": lack - taken, "free_count": count - taken.sum(dtype=torch.int32), "positions": positions.to(torch.int32),
            "slots": slots, "mask": mask if state["parents"] is not None else None}


def _normed(x, gain):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()


def _rotate(x, positions, inv_freq, interleaved):
    """x (tokens, heads, dim) in 32 bits with its leading pairs turned by positions * inv_freq."""
    angle = positions.to(torch.float64)[:, None] * inv_freq
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    r = 2 * inv_freq.numel()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _append(state, case):
    kind, page = DTYPES[case["dtype"]], case["page"]
    seq, index = _places(state["query_start"], state["tokens"])
    position = state["past_lens"][seq].long() + index
    pages, slot = state["block_table"][seq, position // page].long(), position % page
    q = _rotate(_normed(state["q"], state["q_gain"]), position, state["inv_freq"], case["interleaved"]).to(kind)
    k = _rotate(_normed(state["k"], state["k_gain"]), position, state["inv_freq"], case["interleaved"]).to(kind)
    state["k_cache"][0][pages, :, slot] = k
    state["v_cache"][0][pages, :, slot] = state["v"].to(kind)
    return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"]}


def _attend(state, case):
    q, table = state["q"], state["block_table"].long()
    tokens, h, d = q.shape
    hk, seqs = case["kv_heads"], case["seqs"]
    group, most = h // hk, state["most"]
    # keys and values of every sequence, its pages one after the other: (sequences, kv heads, keys, dim)
    k = state["k_cache"][0][table].transpose(1, 2).flatten(2, 3).float()
    v = state["v_cache"][0][table].transpose(1, 2).flatten(2, 3).float()
    start, past = state["query_start"].long(), state["past_lens"].long()
    row = torch.arange(most, device="cuda")
    x = q[(start[:-1, None] + row).clamp(max=tokens - 1)].float()
    x = x.view(seqs, most, hk, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, hk, most * group, d)
    bits = _bits(state["mask"], state["query_start"], most)
    key = torch.arange(k.shape[2], device="cuda")
    before = (key < past[:, None])[:, None, :].expand(-1, most, -1)
    if case["window"]:
        own_bit = bits[:, row, row]
        position = past[:, None] + bits.sum(-1) - own_bit.long()
        before = before & (key > position[..., None] - case["window"])
    drafted = (key[None, :] - past[:, None]).clamp(min=-1, max=bits.shape[2])
    inside = (drafted >= 0) & (drafted < bits.shape[2])
    drafted = drafted.clamp(min=0, max=bits.shape[2] - 1)[:, None, :].expand(-1, most, -1)
    seen = (before | (bits.gather(2, drafted) & inside[:, None, :]))[:, None, :, None, :]
    s = torch.matmul(x, k.transpose(-1, -2).contiguous()).mul_(state["scale"]).view(seqs, hk, most, group, -1)
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hk, most * group, -1), v).view(seqs, hk, most, group, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    seq, index = _places(state["query_start"], tokens)
    return o.permute(0, 2, 1, 3, 4)[seq, index].reshape(tokens, h, d).to(q.dtype)


def _pick(state, case):
    x = state["logits"].float()
    tokens, vocab = x.shape
    seqs = case["seqs"]
    seq, index = _places(state["query_start"], tokens)
    at = torch.arange(state["history"].shape[1], device="cuda")
    there = at < state["past_lens"][:, None]
    answered = there & (at >= state["prompt_lens"][:, None])
    row = torch.arange(seqs, device="cuda")[:, None].expand_as(there)
    counts = torch.zeros((seqs, vocab), device="cuda")
    prompt = torch.zeros((seqs, vocab), dtype=torch.bool, device="cuda")
    counts.index_put_((row[answered], state["history"][answered].long()), torch.ones((), device="cuda"), accumulate=True)
    prompt[row[there & ~answered], state["history"][there & ~answered].long()] = True
    counts, prompt = counts[seq], prompt[seq]
    if case["tree"]:
        bits = _bits(state["mask"], state["query_start"], state["most"])[seq, index]
        who, which = torch.nonzero(bits, as_tuple=True)
        drafted = state["draft"][state["query_start"][seq[who]].long() + which].long()
        counts.index_put_((who, drafted), torch.ones((), device="cuda"), accumulate=True)
    seen = prompt | (counts > 0)
    r, p, f = (state[n][seq][:, None] for n in ("repetition", "presence", "frequency"))
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - f * counts
    x = torch.where(counts > 0, x - p, x)
    if case["biases"]:
        bias = torch.zeros((seqs, vocab), device="cuda")
        of = torch.arange(seqs, device="cuda").repeat_interleave(case["biases"])
        bias[of, state["bias_tokens"].long()] = state["bias_values"]
        x = x + bias[seq]
    if case["grammar"]:
        v = torch.arange(vocab, device="cuda")
        x = torch.where((state["allowed"][:, v // 32] >> (v % 32)) & 1 > 0, x, -math.inf)
    # the lowest index among the largest; -1 where nothing is left
    top = x.amax(-1, keepdim=True)
    v = torch.arange(vocab, device="cuda", dtype=torch.int32)
    best = torch.where(x == top, v, vocab).amin(-1)
    best = torch.where(top[:, 0] > -math.inf, best, -1).to(torch.int32)
    return {"tokens": best, "logits": x if case["out"] else None}


def _settle(state, case):
    tokens, seqs, most, page = state["tokens"], case["seqs"], state["most"], case["page"]
    start, past = state["query_start"], state["past_lens"].long()
    seq, index = _places(start, tokens)
    parents, draft = state["parents"].long(), state["draft"]
    first = start[seq].long()
    # a draft is right if it is what was chosen behind its parent, and no sibling before it is the same
    right = (index == 0) | ((parents >= 0) & (draft == state["choice"][(first + parents.clamp(min=0)).clamp(max=tokens - 1)]))
    grid = torch.full((seqs, most), -2, dtype=torch.int64, device="cuda")
    drafts = grid.clone()
    grid[seq, index], drafts[seq, index] = parents, draft.long()
    twin = (grid[seq] == parents[:, None]) & (drafts[seq] == draft[:, None]) & (torch.arange(most, device="cuda") < index[:, None])
    right &= ~twin.any(-1)
    closure = _ancestors(state["parents"], start, most)[seq, index]
    wrong = torch.zeros((seqs, most), dtype=torch.bool, device="cuda")
    wrong[seq, index] = ~right
    taken = ~(closure & wrong[seq]).any(-1) & closure[:, 0]
    accepted = torch.zeros(seqs, dtype=torch.int64, device="cuda").index_add_(0, seq, taken.long())
    depth = closure.sum(-1) - 1
    path = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    path[first[taken] + depth[taken]] = index[taken].to(torch.int32)
    last = (start[:-1].long() + path[(start[:-1].long() + accepted - 1)].long())
    b, i = seq[taken], index[taken]
    state["history"][b, past[b] + depth[taken]] = draft[taken]
    source, target = past[b] + i, past[b] + depth[taken]
    table = state["block_table"].long()
    for cache in (state["k_cache"], state["v_cache"]):
        moved = cache[:, table[b, source // page], :, source % page]
        cache[:, table[b, target // page], :, target % page] = moved
    return {"accepted": accepted.to(torch.int32), "tokens": state["choice"][last], "path": path,
            "lens": (past + accepted).to(torch.int32), "history": state["history"],
            "k_cache": state["k_cache"], "v_cache": state["v_cache"]}


def exact(case, seed):
    """What `run` returns where it computes numbers, in 64 bits, one sequence and head after the other."""
    state = prepare(case, seed)
    op = case["op"]
    new, past = lengths(case)
    if op == "assign" or (op == "logits" and not case["out"]):
        return None
    if op == "settle":
        return _settle_exact(state, case, new, past)
    if op == "norm":
        return _turn_exact(_norm_exact(state["x"], state["q_gain"]), state["positions"].double(), case)
    first = [sum(new[:b]) for b in range(case["seqs"] + 1)]
    if op == "logits":
        return {"tokens": None, "logits": _logits_exact(state, case, first, past)}
    page, d = case["page"], case["head_dim"]
    if op == "append":
        at = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, past)])
        q = _turn_exact(_norm_exact(state["q"], state["q_gain"]), at.double(), case)
        k = _turn_exact(_norm_exact(state["k"], state["k_gain"]), at.double(), case)
        caches = state["k_cache"].double(), state["v_cache"].double()
        for b in range(case["seqs"]):
            part = slice(first[b], first[b + 1])
            slot = state["block_table"][b].long().index_select(0, at[part] // page) * page + at[part] % page
            for cache, rows in zip(caches, (k[part], state["v"][part].double())):
                flat = cache[0].permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], d)
                flat.index_copy_(0, slot, rows)
                cache[0].copy_(flat.view(-1, page, case["kv_heads"], d).permute(0, 2, 1, 3))
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    parents = state["parents"].tolist()
    for b in range(case["seqs"]):
        n, p = new[b], past[b]
        chain = [[i] for i in range(n)]
        for i in range(n):
            if parents[first[b] + i] >= 0:
                chain[i] = chain[parents[first[b] + i]] + [i]
        seen = torch.ones((n, p + n), dtype=torch.bool)
        seen[:, p:] = False
        for i in range(n):
            seen[i, torch.tensor(chain[i]) + p] = True
            if case["window"]:
                seen[i, : max(0, min(p, p + len(chain[i]) - 1 - case["window"] + 1))] = False
        seen = seen.cuda()
        pos = torch.arange(p + n, device="cuda")
        pages = state["block_table"][b].long()[pos // page]
        for hk in range(case["kv_heads"]):
            k, v = (state[c][0][pages, hk, pos % page].double() for c in ("k_cache", "v_cache"))
            x = state["q"][first[b] : first[b + 1], hk * group : (hk + 1) * group].double()
            s = (x.reshape(n * group, d) @ k.T * state["scale"]).view(n, group, -1)
            w = torch.softmax(s.masked_fill(~seen[:, None, :], -math.inf), -1)
            out[first[b] : first[b + 1], hk * group : (hk + 1) * group] = (w.view(n * group, -1) @ v).view(n, group, d)
    return out


def _norm_exact(x, gain):
    x = x.double()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * gain.double()


def _turn_exact(x, position, case):
    """The pairs as complex numbers, multiplied by exp(i * angle)."""
    half = case["rot_dim"] // 2
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


def _settle_exact(state, case, new, past):
    """The caches alone: each sequence's tree walked from its first token, the nodes met moved one after the other."""
    caches = state["k_cache"].double(), state["v_cache"].double()
    parents, draft, choice, table = (state[n].tolist() for n in ("parents", "draft", "choice", "block_table"))
    first, page = 0, case["page"]
    for b in range(case["seqs"]):
        node, place = 0, past[b]
        while True:
            after = [i for i in range(node + 1, new[b]) if parents[first + i] == node and draft[first + i] == choice[first + node]]
            if not after:
                break
            node, place = after[0], place + 1
            source = past[b] + node
            for cache in caches:
                cache[:, table[b][place // page], :, place % page] = cache[:, table[b][source // page], :, source % page]
        first += new[b]
    return {"accepted": None, "tokens": None, "path": None, "lens": None, "history": None, "k_cache": caches[0], "v_cache": caches[1]}


def _logits_exact(state, case, first, past):
    """Row by row: the tokens a row has behind it, counted by value."""
    x = state["logits"].double()
    vocab = case["vocab"]
    words = None if state["mask"] is None else state["mask"].cpu()
    for b in range(case["seqs"]):
        r, p, f = (float(state[n][b]) for n in ("repetition", "presence", "frequency"))
        text = state["history"][b, : past[b]].long()
        prompt = text[: int(state["prompt_lens"][b])]
        for t in range(first[b], first[b + 1]):
            answer = text[int(state["prompt_lens"][b]) :]
            if words is not None:
                nodes = [j for j in range(first[b + 1] - first[b]) if (int(words[t, j // 64]) >> (j % 64)) & 1]
                answer = torch.cat((answer, state["draft"][[first[b] + j for j in nodes]].long()))
            number = torch.bincount(answer, minlength=vocab).double()
            seen = (number + torch.bincount(prompt, minlength=vocab)) > 0
            row = x[t]
            row = torch.where(seen & (row > 0), row / r, torch.where(seen, row * r, row)) - f * number - p * (number > 0)
            if case["biases"]:
                part = slice(b * case["biases"], (b + 1) * case["biases"])
                row[state["bias_tokens"][part].long()] += state["bias_values"][part].double()
            if case["grammar"]:
                v = torch.arange(vocab, device="cuda")
                row[((state["allowed"][t].long()[v // 32] >> (v % 32)) & 1) == 0] = -math.inf
            x[t] = row
    return x

"""A step of greedy decoding with drafted trees, its operators one after the other as a program calls them, eager and as
one captured graph: tables from lengths, norms and append, attention over the tree, logits under rules, the path, and
the cache closed up behind it.  The text that comes out has to be the one that plain steps of one token give."""
import numpy as np
import pytest
import torch

import step_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu
HQ, HK, D, PAGE, VOCAB, LAYERS, NODES, SEQS, COLUMNS = 8, 2, 64, 8, 501, 2, 12, 3, 30


class Model:
    """Layers of norms, attention and a projection, between an embedding and its transpose, from a seed."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        self.embed = n(VOCAB, HQ * D)
        self.qkv = [n(HQ * D, (HQ + 2 * HK) * D) * 0.05 for _ in range(LAYERS)]
        self.o = [n(HQ * D, HQ * D) * 0.05 for _ in range(LAYERS)]
        self.gains = [(1 + 0.1 * n(D), 1 + 0.1 * n(D)) for _ in range(LAYERS)]


class Server:
    def __init__(self, q4, model, tokens, words):
        self.q4, self.m, self.tokens = q4, model, tokens
        pages = SEQS * COLUMNS
        self.caches = [q4.KVCache(*(torch.zeros(pages, HK, PAGE, D, dtype=torch.float16, device="cuda") for _ in range(2))) for _ in range(LAYERS)]
        self.layers = q4.KVLayers(self.caches)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.held = torch.full((SEQS, COLUMNS), -1, **i32), torch.zeros(SEQS, **i32)
        self.free_count = torch.full((1,), pages, **i32)
        self.free = torch.randperm(pages, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.int32)
        self.step = q4.KVStep(SEQS, COLUMNS, PAGE, tokens, words, max_query_len=tokens, max_context_len=COLUMNS * PAGE)
        self.history, self.past = torch.zeros(SEQS, COLUMNS * PAGE, **i32), torch.zeros(SEQS, **i32)
        self.prompt, self.new = torch.zeros(SEQS, **i32), torch.zeros(SEQS, **i32)
        self.draft, self.parents = torch.zeros(tokens, **i32), torch.full((tokens,), -1, **i32)
        self.freq, _ = q4.rope_frequencies(D, 1e4)
        self.rules = q4.LogitRules(query_start=self.step.query_start, history=self.history, history_lens=self.past, prompt_lens=self.prompt,
                                   draft=self.draft, mask=self.step.mask, repetition=torch.full((SEQS,), 1.3, device="cuda"),
                                   frequency=torch.full((SEQS,), 0.4, device="cuda"), presence=torch.full((SEQS,), 0.2, device="cuda"))

    def forward(self):
        q4, s, m = self.q4, self.step, self.m
        q4.q4_kv_assign(s, self.table, self.held, self.past, self.new, self.free, self.free_count, parents=self.parents)
        x = m.embed[self.draft.long().clamp(0, VOCAB - 1)]
        for i, cache in enumerate(self.caches):
            q, k, v = (x @ m.qkv[i]).view(self.tokens, -1, D).split([HQ, HK, HK], 1)
            q = q4.q4_kv_append_norm(cache, s.batch, k, v, q=q, k_gain=m.gains[i][1], q_gain=m.gains[i][0], inv_freq=self.freq, positions=s.positions)
            x = x + q4.q4_attention_tree(cache, s.batch, q, s.mask).view(self.tokens, -1).float() @ m.o[i]
        self.logits = x @ m.embed.T * 0.05
        self.choice = q4.q4_logits_argmax(self.logits, self.rules)
        self.accepted, self.next, self.path, lens = q4.q4_tree_accept(s.batch, self.choice, self.draft, parents=self.parents, history=self.history)
        q4.q4_kv_move(self.layers, s.batch, self.path, self.accepted)
        # the next step's inputs
        self.table.copy_(s.block_table)
        self.held.copy_(s.held)
        self.free_count.copy_(s.free_count)
        self.past.copy_(lens)

    def load(self, rows):
        """(tokens, parents) of each sequence."""
        self.new.copy_(torch.tensor([len(t) for t, _ in rows], dtype=torch.int32))
        flat, par = [x for t, _ in rows for x in t], [x for _, p in rows for x in p]
        pad = self.tokens - len(flat)
        self.draft.copy_(torch.tensor(flat + [0] * pad, dtype=torch.int32))
        self.parents.copy_(torch.tensor(par + [-1] * pad, dtype=torch.int32))


def text_of_plain_steps(q4, model, prompts, steps):
    """One token a sequence and step: each sequence's picks."""
    plain = Server(q4, model, 40, 1)
    plain.load([(p, list(range(-1, len(p) - 1))) for p in prompts])
    plain.prompt.copy_(torch.tensor([len(p) for p in prompts], dtype=torch.int32))
    texts = [[] for _ in prompts]
    # the prompts as chains of which everything is accepted: their drafts are what was chosen, by decree
    accept = q4.q4_tree_accept

    def all_of_it(batch, choice, draft, parents=None, history=None):
        got = accept(batch, choice, draft, parents=parents, history=history)
        start = batch._keep[1].tolist()
        for b in range(SEQS):
            n = start[b + 1] - start[b]
            got[0][b], got[1][b], got[3][b] = n, choice[start[b + 1] - 1], batch._keep[2][b]
            history[b, int(got[3][b]) - n : int(got[3][b])] = draft[start[b] : start[b + 1]]
            got[2][start[b] : start[b + 1]] = torch.arange(n, dtype=torch.int32)
        return got

    q4.q4_tree_accept = all_of_it
    try:
        plain.forward()
    finally:
        q4.q4_tree_accept = accept
    after = [x.clone() for x in (plain.table, plain.held, plain.free_count, plain.past, plain.history)], [(c.k.clone(), c.v.clone()) for c in plain.caches]
    first = plain.next.tolist()
    margins = []
    tokens = list(first)
    for _ in range(steps):
        plain.load([([t], [-1]) for t in tokens])
        plain.forward()
        texts = [x + [t] for x, t in zip(texts, tokens)]
        tokens = plain.next.tolist()
    return texts, first, after, margins


@pytest.mark.parametrize("captured", [False, True])
def test_trees_give_the_plain_text(captured):
    """Trees whose branches are right now and then: every token taken is the one that plain decoding picks, and the cache,
    closed up, serves the next step."""
    q4 = lib()
    say("tree steps", captured)
    model = Model(4)
    prompts = [[5, 9, 200, 7], [3] * 11, [1, 2]]
    texts, first, (state, caches), _ = text_of_plain_steps(q4, model, prompts, 40)
    server = Server(q4, model, SEQS * NODES + 2, 1)
    for own, was in zip((server.table, server.held, server.free_count, server.past, server.history), state):
        own.copy_(was)
    for c, (k, v) in zip(server.caches, caches):
        c.k.copy_(k)
        c.v.copy_(v)
    server.prompt.copy_(torch.tensor([len(p) for p in prompts], dtype=torch.int32))
    rng = np.random.default_rng(2)
    done, cur = [0] * SEQS, list(first)
    graph = None
    if captured:
        kept = [x.clone() for x in (server.table, server.held, server.free_count, server.past, server.history)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            server.forward()  # no new tokens: nothing is written
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            server.forward()
        for own, was in zip((server.table, server.held, server.free_count, server.past, server.history), kept):
            own.copy_(was)
    taken = 0
    for _ in range(12):
        rows = []
        for b in range(SEQS):
            if done[b] > 25:
                rows.append(([], []))
                continue
            n = int(rng.integers(1, NODES + 1))
            parents = step_ref.tree(n, rng)
            tokens = [cur[b]] + [0] * (n - 1)
            depth = [0] * n
            right = [True] + [False] * (n - 1)
            for i in range(1, n):
                p = parents[i]
                depth[i] = depth[p] + 1
                right[i] = right[p] and rng.random() < 0.7
                tokens[i] = texts[b][done[b] + depth[i]] if right[i] else int(rng.integers(0, VOCAB))
            rows.append((tokens, parents))
        server.load(rows)
        if graph:
            graph.replay()
        else:
            server.forward()
        torch.cuda.synchronize()
        accepted, following = server.accepted.tolist(), server.next.tolist()
        assert server.step.missing.tolist() == [0] * SEQS
        for b in range(SEQS):
            n = accepted[b]
            assert (n > 0) == bool(rows[b][0])
            if not n:
                continue
            at = len(prompts[b]) + done[b]
            got = server.history[b, at : at + n].tolist()
            assert got == texts[b][done[b] : done[b] + n], (b, done[b])
            done[b] += n
            cur[b] = following[b]
            assert cur[b] == texts[b][done[b]]
            assert int(server.past[b]) == at + n
            taken += n
    assert taken > 36  # more than one token a sequence and step


def test_a_sequence_without_pages_touches_no_other():
    """A sequence whose pages do not fit, with others' pages behind its own in the row: keys, values, outputs and moves of
    the others are as without it, its own tokens are not stored."""
    q4 = lib()
    page, hq, hk, dim = 16, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = (torch.randn(9, hk, page, dim, device="cuda", generator=g).half() for _ in range(2))
    x = torch.randn(12, hq + 2 * hk, dim, device="cuda", generator=g)
    parents = [-1, 0, 0, 1, -1, 0, 0, 1, -1, 0, 1, 1]
    draft, choice = i32([7, 1, 2, 3] * 3), i32([2, 9, 5, 9, 2, 9, 5, 9, 1, 2, 9, 9])
    freq, _ = q4.rope_frequencies(dim)
    got = []
    for news in ([4, 4, 4], [4, 0, 4]):
        caches = k.clone(), v.clone()
        cache = q4.KVCache(*caches)
        step = q4.KVStep(3, 4, page, 12, 1)
        # the second needs another page, none is left; behind its own stand the first's and the third's
        table = i32([[0, 1, 8, 8], [2, 0, 1, 5], [4, 5, 0, 0]])
        rows = [0, 1, 2, 3] + ([4, 5, 6, 7] if news[1] else []) + [8, 9, 10, 11]
        pad = 12 - len(rows)
        pick = torch.tensor(rows + [0] * pad, device="cuda")
        own = torch.tensor([parents[r] for r in rows] + [-1] * pad, dtype=torch.int32, device="cuda")
        q4.q4_kv_assign(step, table, i32([2, 1, 2]), i32([20, 14, 17]), i32(news), i32([7]), i32([0]), parents=own)
        q, kk, vv = x[pick].split([hq, hk, hk], 1)
        turned = q4.q4_kv_append_norm(cache, step.batch, kk, vv, q=q, inv_freq=freq, positions=step.positions)
        out = q4.q4_attention_tree(cache, step.batch, turned, step.mask)
        accepted, following, path, lens = q4.q4_tree_accept(step.batch, choice[pick].contiguous(), draft[pick].contiguous(), parents=own)
        q4.q4_kv_move(cache, step.batch, path, accepted)
        torch.cuda.synchronize()
        at = [i for i, r in enumerate(rows) if r < 4 or r >= 8]
        got.append((step, accepted, caches, out[at].clone()))
    full, without = got
    assert full[0].missing.tolist() == [0, 1, 0] and full[0].block_table.tolist()[1] == [2, -1, 1, 5]
    assert full[0].slots[4:8].tolist() == [2 * page + 14, 2 * page + 15, -1, -1]
    assert [full[1].tolist()[b] for b in (0, 2)] == [without[1].tolist()[b] for b in (0, 2)]
    assert torch.equal(full[3], without[3])
    for a, b, was in zip(full[2], without[2], (k, v)):
        others = [p for p in range(9) if p != 2]
        assert torch.equal(a[others], b[others])
        assert torch.equal(a[2, :, :14], was[2, :, :14])  # its own page: the two tokens that have a place


def test_each_on_a_stream_of_its_own():
    """Every operator on a stream that is not the current one, behind work there that makes its inputs."""
    q4 = lib()
    g = torch.Generator(device="cuda").manual_seed(3)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    freq, _ = q4.rope_frequencies(128)
    table, start, ctx = i32([[3, 1, 0], [2, 5, 4]]), i32([0, 5, 9]), i32([40, 44])
    batch = q4.KVBatch(table, start, ctx)
    x = torch.randn(9, 12, 128, device="cuda", generator=g).half()
    base = [torch.randn(6, 2, 16, 128, device="cuda", generator=g).half() for _ in range(2)]
    mask = torch.tensor([1, 3, 7, 11, 19, 1, 3, 7, 15], device="cuda").view(9, 1)
    logits = torch.randn(9, 30000, device="cuda", generator=g)
    history = torch.randint(0, 30000, (2, 50), device="cuda", generator=g, dtype=torch.int32)
    pos = i32(range(9))

    def norm(x, stream=None):
        return [q4.q4_norm_rope(x, None, 1e-6, pos, freq, stream=stream)]

    def append(x, stream=None):
        kv = [t.clone() for t in base]
        torch.cuda.synchronize()
        q, k, v = x.split([8, 2, 2], 1)
        return [q4.q4_kv_append_norm(q4.KVCache(*kv), batch, k, v, q=q, inv_freq=freq, stream=stream)] + kv

    def tree(x, stream=None):
        return [q4.q4_attention_tree(q4.KVCache(*base), batch, x, mask, stream=stream)]

    def pick(x, stream=None):
        rules = q4.LogitRules(query_start=start, history=history, history_lens=i32([50, 20]), presence=torch.ones(2, device="cuda"))
        torch.cuda.synchronize()
        return [q4.q4_logits_argmax(x, rules, stream=stream)]

    def assign(x, stream=None):
        step = q4.KVStep(2, 3, 16, 9, 1)
        left, count = i32([9, 8, 7, 6]), i32([4])
        torch.cuda.synchronize()
        q4.q4_kv_assign(step, table, x[0], x[1], x[2], left, count, stream=stream)
        return [step.block_table, step.held, step.missing, step.slots, step.mask]

    def accept(x, stream=None):
        return list(q4.q4_tree_accept(batch, x[0], x[1], parents=x[2], stream=stream))

    def move(x, stream=None):
        kv = [t.clone() for t in base]
        torch.cuda.synchronize()
        q4.q4_kv_move(q4.KVCache(*kv), batch, x[:9], x[9:], stream=stream)
        return kv

    cases = ((norm, x), (append, x), (tree, x[:, :8].contiguous()), (pick, logits), (assign, i32([[1, 2], [16, 30], [5, 4]])),
             (accept, i32([[4, 9, 1, 1, 3, 5, 5, 5, 5], [0, 4, 7, 9, 8, 0, 5, 5, 5], [-1, 0, 0, 1, 1, -1, 0, 1, 2]])),
             (move, i32([0, 2, 4, -1, -1, 0, 3, -1, -1, 3, 2])))
    side, slow = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda").half()
    for fn, real in cases:
        say("stream", fn.__name__)
        want = fn(real)
        given = torch.zeros_like(real)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                slow @ slow
            given.copy_(real)
        got = fn(given, stream=side)
        side.synchronize()
        if fn is append or fn is move or fn is assign or fn is pick:
            torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), fn.__name__

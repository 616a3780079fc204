"""Steps with drafted trees that run out of pages, or reach the end of their block table: the text goes on where keys and
values could be stored and stands still otherwise, and what comes out is the text of plain steps."""
import numpy as np
import pytest
import torch

import step_ref
import test_gpu_tree_step as tree_step
from gpu_util import lib, say

pytestmark = pytest.mark.gpu
PROMPTS = [[5, 9, 200, 7], [3] * 11, [1, 2]]
STEPS = 42


def made_model():
    """A model whose layers outweigh a token's own embedding, so that its text depends on what the cache holds (18 or more
    tokens among 42; each pick is 1.3 above the next)."""
    model = tree_step.Model(10)
    for o in model.o:
        o *= 30
    return model


def server_behind(q4, model, state, caches, captured):
    """A Server with the prompts behind it, pages that nobody holds full of what a former owner left, and its step as a
    function."""
    server = tree_step.Server(q4, model, tree_step.SEQS * tree_step.NODES + 2, 1)
    own = (server.table, server.held, server.free_count, server.past, server.history)
    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            server.forward()  # no new tokens
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            server.forward()
    for t, was in zip(own, state):
        t.copy_(was)
    g = torch.Generator(device="cuda").manual_seed(7)
    held = torch.zeros(server.free.shape[0], dtype=torch.bool, device="cuda")
    for b in range(tree_step.SEQS):
        held[server.table[b, : int(server.held[b])].long()] = True
    for c, (k, v) in zip(server.caches, caches):
        for t, was in ((c.k, k), (c.v, v)):
            t.copy_(torch.where(held[:, None, None, None], was, 3 * torch.randn(was.shape, device="cuda", generator=g).half()))
    server.prompt.copy_(torch.tensor([len(p) for p in PROMPTS], dtype=torch.int32))
    return server, graph.replay if graph else server.forward


def trees(rng, texts, done, cur):
    """A tree for each sequence whose branches are right now and then."""
    rows = []
    for text, at, token in zip(texts, done, cur):
        n = int(rng.integers(6, tree_step.NODES + 1))
        parents = step_ref.tree(n, rng)
        tokens, depth, right = [token] + [0] * (n - 1), [0] * n, [True] + [False] * (n - 1)
        for i in range(1, n):
            p = parents[i]
            depth[i] = depth[p] + 1
            right[i] = right[p] and rng.random() < 0.8 and at + depth[i] < len(text)
            tokens[i] = text[at + depth[i]] if right[i] else int(rng.integers(0, tree_step.VOCAB))
        rows.append((tokens, parents))
    return rows


def settle(server, texts, done, cur):
    """What the step took of each sequence, which has to be its text."""
    torch.cuda.synchronize()
    took, past = server.accepted.tolist(), server.past.tolist()
    for b, n in enumerate(took):
        at = len(PROMPTS[b]) + done[b]
        assert past[b] == at + n, (b, past[b], at, n)
        assert server.history[b, at : at + n].tolist() == texts[b][done[b] : done[b] + n], (b, done[b])
        done[b] += n
        cur[b] = server.next.tolist()[b]
        assert cur[b] == texts[b][done[b]], b  # without a token taken: the same one again
    return took


@pytest.mark.parametrize("captured", [False, True])
def test_pages_run_out_and_come_back(captured):
    """Now and then no page is left: sequences that need one stand still (or go on in the page they hold), the others go on;
    once there are pages again all have their text."""
    q4 = lib()
    say("pages run out", captured)
    model = made_model()
    texts, first, (state, caches), _ = tree_step.text_of_plain_steps(q4, model, PROMPTS, STEPS)
    server, step = server_behind(q4, model, state, caches, captured)
    rng = np.random.default_rng(5)
    done, cur = [0] * tree_step.SEQS, list(first)
    # no page at all: to the end of the pages that the prompts began, and no further
    free = int(server.free_count)
    server.free_count.zero_()
    for turn in range(12):
        server.load(trees(rng, texts, done, cur))
        step()
        took = settle(server, texts, done, cur)
    ends = [-len(p) % tree_step.PAGE for p in PROMPTS]
    assert (done, took, min(server.step.missing.tolist()) > 0) == (ends, [0] * tree_step.SEQS, True)
    server.free_count.fill_(free)
    lacked = 0
    for turn in range(24):
        if max(done) > 26:
            break
        server.load(trees(rng, texts, done, cur))
        free = int(server.free_count)
        starved = turn % 3 != 2
        if starved:
            server.free_count.zero_()
        step()
        took = settle(server, texts, done, cur)
        missing = server.step.missing.tolist()
        assert starved or missing == [0] * tree_step.SEQS
        lacked += sum(m > 0 for m in missing)
        assert all(m > 0 for m, n in zip(missing, took) if n == 0)
        if starved:
            server.free_count.fill_(free)
    assert lacked > 5 and min(done) > 8


@pytest.mark.parametrize("captured", [False, True])
def test_the_end_of_the_table(captured, monkeypatch):
    """Sequences that grow to the last place of their row of the table, the trees' last nodes behind it, and stand still
    there."""
    q4 = lib()
    say("end of the table", captured)
    model = made_model()
    texts, first, _, _ = tree_step.text_of_plain_steps(q4, model, PROMPTS, STEPS)
    monkeypatch.setattr(tree_step, "COLUMNS", 5)
    end = 5 * tree_step.PAGE
    _, again, (state, caches), _ = tree_step.text_of_plain_steps(q4, model, PROMPTS, 0)
    assert again == first
    server, step = server_behind(q4, model, state, caches, captured)
    rng = np.random.default_rng(9)
    done, cur = [0] * tree_step.SEQS, list(first)
    for _ in range(60):
        server.load(trees(rng, texts, done, cur))
        step()
        took = settle(server, texts, done, cur)
        assert server.step.missing.tolist() == [0] * tree_step.SEQS
        for b in range(tree_step.SEQS):
            assert took[b] or len(PROMPTS[b]) + done[b] == end
    assert [len(p) + d for p, d in zip(PROMPTS, done)] == [end] * tree_step.SEQS


def walk(start, ctx, choice, draft, parents, slots, tokens, history):
    """As step_ref.accept, of the nodes that have a slot."""
    accepted, following, lens, path = [], [], [], [None] * tokens
    for b in range(len(ctx)):
        first, last = int(start[b]), int(start[b + 1])
        n = 0 if first < 0 or last > tokens or last < first else last - first
        past = int(ctx[b]) - max(last - first, 0)
        got = [0] if n and slots[first] >= 0 else []
        while got:
            cur, want = got[-1], int(choice[first + got[-1]])
            after = [i for i in range(cur + 1, n) if (i - 1 if parents is None else int(parents[first + i])) == cur
                     and int(draft[first + i]) == want and want >= 0 and slots[first + i] >= 0]
            if not after:
                break
            got.append(after[0])
        for j in range(n):
            path[first + j] = got[j] if j < len(got) else -1
        for j, i in enumerate(got):
            if 0 <= past + j < history.shape[1]:
                history[b, past + j] = draft[first + i]
        accepted.append(len(got))
        following.append(int(choice[first + got[-1]]) if got else int(draft[first]) if n else -1)
        lens.append(past + len(got))
    return accepted, following, path, lens


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("new", [[1], [16, 0, 3], [64, 65, 1, 9], [200, 300, 256, 257, 5], [1000, 7]])
def test_nodes_without_a_slot(new, chain):
    """Paths of nodes that have slots only: none at all, from some node on, and any of them without one."""
    q4 = lib()
    i32 = lambda x: torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")  # noqa: E731
    for seed in range(6):
        rng = np.random.default_rng(seed)
        parents, choice, draft, slots = [], [], [], []
        for n in new:
            p = [i - 1 for i in range(n)] if chain else step_ref.tree(n, rng)
            c, d = rng.integers(0, 4, n), rng.integers(0, 4, n)
            for i in range(1, n):
                if p[i] >= 0 and rng.random() < 0.9:
                    d[i] = c[p[i]]
            s = rng.integers(0, 2 ** 40, n)
            if seed % 3 == 0:
                s[int(rng.integers(0, n + 1)):] = -1
            elif seed % 3 == 1:
                s[rng.random(n) < 0.2] = -1
            elif n:
                s[0] = -1
            parents, choice, draft, slots = parents + list(p), choice + list(c), draft + list(d), slots + list(s)
        tokens, pad = sum(new) + 2, [1, 1]
        start = np.concatenate([[0], np.cumsum(new)])
        ctx = [n + int(rng.integers(0, 40)) for n in new]
        history = rng.integers(0, 9, (len(new), max(ctx))).astype(np.int32)
        batch = q4.KVBatch(torch.zeros(len(new), 1, dtype=torch.int32, device="cuda"), i32(start), i32(ctx))
        text = torch.from_numpy(history).cuda()
        out = tuple(torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (len(new), len(new), tokens, len(new)))
        say("slots", new, chain, seed)
        got = q4.q4_tree_accept(batch, i32(choice + pad), i32(draft + pad), parents=None if chain else i32(parents + pad), history=text, out=out,
                                slots=torch.tensor([int(x) for x in slots + pad], device="cuda"))
        want = walk(start, ctx, choice, draft, None if chain else parents, slots, tokens, history)
        torch.cuda.synchronize()
        assert [x.tolist() for x in got[:2]] == [want[0], want[1]] and got[3].tolist() == want[3]
        assert got[2].tolist() == [-77 if x is None else x for x in want[2]]
        assert np.array_equal(text.cpu().numpy(), history)


def test_slots_of_a_step():
    """The batch of a KVStep brings its slots; rows behind the step's are of no sequence."""
    q4 = lib()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    step = q4.KVStep(2, 2, 16, 8, 1)
    parents = [-1, 0, 1, -1, 0, 1]
    # the second needs a page for its last two tokens, none is left
    q4.q4_kv_assign(step, i32([[0, 5], [1, 6]]), i32([1, 1]), i32([3, 15]), i32([3, 3]), i32([9]), i32([0]), parents=i32(parents + [-1, -1]))
    for more in (0, 3):
        pad = [-1] * (2 + more)
        choice, draft = i32([4, 5, 6, 7, 8, 9] + pad), i32([3, 4, 5, 2, 7, 8] + pad)
        text = torch.zeros(2, 32, dtype=torch.int32, device="cuda")
        accepted, following, path, lens = q4.q4_tree_accept(step.batch, choice, draft, parents=i32(parents + pad), history=text)
        assert (accepted.tolist(), following.tolist(), path.tolist()[:6], lens.tolist()) == ([3, 1], [6, 7], [0, 1, 2, 0, -1, -1], [6, 16])
        assert text[0, 3:6].tolist() == [3, 4, 5] and text[1].tolist() == [0] * 15 + [2] + [0] * 16
    with pytest.raises(ValueError):
        q4.q4_tree_accept(step.batch, choice, draft, slots=step.slots)  # fewer slots than rows
    with pytest.raises(TypeError):
        q4.q4_tree_accept(step.batch, choice[:8], draft[:8], slots=i32([0] * 8))


def test_a_new_step_has_no_slots():
    """Rows that no step wrote yet name no place of the cache (0 is one), also where the first steps are shorter."""
    q4 = lib()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for words in (0, 1, 3):
        step = q4.KVStep(2, 2, 16, 9, words)
        assert step.slots.tolist() == [-1] * 9 and step.positions.tolist() == [0] * 9
        assert words == 0 or not step.mask.any()
        q4.q4_kv_assign(step, i32([[0, 5], [1, 6]]), i32([1, 1]), i32([3, 0]), i32([2, 1]), i32([9]), i32([1]))
        assert step.slots.tolist() == [3, 4, 16] + [-1] * 6

"""q4_kv_assign: block tables, slots, positions and masks from lengths, against the same one sequence after the other on
the host; every output whole, rows that belong to no sequence as they were."""
import numpy as np
import pytest
import torch

import step_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def inputs(past, new, page, columns, seed, spare=3, held=None):
    """A table in which each sequence holds the pages of what it has, others' pages and -1 behind them, and the free
    pages."""
    rng = np.random.default_rng(seed)
    seqs = len(past)
    held = np.array([min(-(-max(p, 0) // page), columns) for p in past] if held is None else held, dtype=np.int32)
    ids = rng.permutation(seqs * columns + spare).astype(np.int32)
    table = rng.integers(-1, seqs * columns, (seqs, columns)).astype(np.int32)
    at = 0
    for b in range(seqs):
        n = min(max(int(held[b]), 0), columns)
        table[b, :n] = ids[at : at + n]
        at += n
    return table, held, ids[at:].copy()


def check(q4, past, new, page, columns, tokens, parents=None, words=0, count=None, held=None, seed=0, in_place=False, stream=None):
    table, held, free = inputs(past, new, page, columns, seed, held=held)
    count = len(free) if count is None else count
    want = step_ref.assign(table, held, past, new, free, count, page, tokens, parents, words)
    dev = [torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda() for x in (table, held, past, new, free, [count])]
    step = q4.KVStep(len(past), columns, page, tokens, words, table=dev[0] if in_place else None)
    if not in_place:
        step.block_table.fill_(-77)
    for t in (step.held, step.query_start, step.context_lens, step.missing, step.free_count, step.positions, step.slots) + ((step.mask,) if words else ()):
        t.fill_(-77)
    q4.q4_kv_assign(step, *dev, parents=None if parents is None else torch.tensor(parents, dtype=torch.int32, device="cuda"), stream=stream)
    torch.cuda.synchronize()
    assert np.array_equal(step.block_table.cpu().numpy(), want["table"])
    for got, name in ((step.held, "held"), (step.query_start, "start"), (step.context_lens, "ctx"), (step.missing, "missing")):
        assert got.tolist() == [int(x) for x in want[name]], name
    assert step.free_count.tolist() == [want["free"]]
    for got, name in ((step.positions, "positions"), (step.slots, "slots")):
        assert got.tolist() == [-77 if x is None else int(x) for x in want[name]], name
    if words:
        assert step.mask.tolist() == [[-77] * words if x is None else x for x in want["mask"]]
    if not in_place:
        assert np.array_equal(dev[0].cpu().numpy(), table)
    return step


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("past,new,page,columns,count", [
    ([0], [1], 16, 1, None), ([0], [0], 8, 1, 0), ([16], [1], 16, 2, None), ([15], [1], 16, 2, None),
    ([5, 0, 31, 100], [1, 0, 1, 40], 16, 10, None), ([5, 0, 31, 100], [30, 17, 1, 40], 16, 10, 3), ([1, 1, 1], [40, 0, 40], 24, 4, 1),
    ([7, 9], [60, 60], 8, 5, None),  # longer than a row of the table
    ([3] * 70, [1] * 70, 64, 3, None), ([0, 8], [500, 700], 40, 40, None), ([0] * 9, [17] * 9, 16, 2, 9),
])
def test_lengths(past, new, page, columns, count, in_place):
    q4 = lib()
    say("assign", past[:4], new[:4], page, columns, count)
    check(q4, past, new, page, columns, sum(new) + 3, count=count, in_place=in_place)


def test_many_sequences():
    """More sequences than workgroups, ragged, and pages for some of them only."""
    q4 = lib()
    rng = np.random.default_rng(1)
    for seqs, count in ((513, None), (1500, 900), (3001, 1)):
        past, new = rng.integers(0, 60, seqs), rng.integers(0, 5, seqs)
        check(q4, past, new, 8, 9, int(new.sum()) + 5, count=count)


def test_long_prompts():
    """Tokens of one sequence over many workgroups, and a table of many pages."""
    q4 = lib()
    check(q4, [3], [50000], 16, 4000, 50001)
    check(q4, [100, 0], [1, 9000], 8, 20000, 9001)


@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("words", [0, 1, 2, 4, 16])
def test_trees(kind, words):
    """Depths and ancestors, of trees larger than the masks too."""
    q4 = lib()
    rng = np.random.default_rng(words)
    new = [1, 0, 16, 64, 65, 130, 7] + ([300] if words in (2, 4) else []) + ([1030] if words in (0, 16) else [])
    parents = [p for n in new for p in step_ref.tree(n, rng, kind)]
    check(q4, list(rng.integers(0, 90, len(new))), new, 16, 80, sum(new) + 4, parents=parents + [0] * 4, words=words)


def test_masks_of_chains():
    """Masks without parents: each token sees those before it."""
    q4 = lib()
    check(q4, [5, 0, 8], [3, 64, 200], 16, 20, 270, words=2)
    check(q4, [5], [1024], 16, 70, 1024, words=16)


def test_parents_that_are_none():
    """A parent that is the node itself, a later one, negative or far away counts as none."""
    q4 = lib()
    parents = [3, 1, 0, 9, 2 ** 31 - 1, -5, 4, 5, -2 ** 31, 8]
    check(q4, [10, 4], [6, 4], 16, 3, 10, parents=parents, words=1)


def test_lengths_out_of_range():
    """Negative lengths count as 0, a held count behind the table as the table, a free count behind the list as the list,
    rows behind `tokens` are not written."""
    q4 = lib()
    check(q4, [-5, 3, 0], [2, -7, 9], 16, 2, 6)
    check(q4, [3, 50], [1, 9], 16, 3, 10, held=[99, -1])
    check(q4, [3, 50], [1, 9], 16, 4, 10, count=1 << 30)
    check(q4, [3, 50], [1, 9], 16, 4, 10, count=-3)
    check(q4, [0, 0, 5], [20, 30, 40], 16, 8, 33)
    check(q4, [2 ** 31 - 1, 1], [2 ** 31 - 1, 3], 16, 2, 4)


def test_tables_in_turn():
    """Steps whose last tables are the next one's inputs, on a stream of its own, and the captured pair replayed."""
    q4 = lib()
    page, columns, tokens = 8, 6, 12
    past, news = [0, 0, 0], [[3, 5, 1], [1, 1, 1], [4, 0, 4], [1, 2, 3]]
    table, held, free = inputs(past, news[0], page, columns, 5)
    stream = torch.cuda.Stream()
    for captured in (False, True):
        steps = [q4.KVStep(3, columns, page, tokens) for _ in range(2)]
        new, lens = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
        fixed = torch.from_numpy(free).cuda()

        def pair():
            q4.q4_kv_assign(steps[1], steps[0].block_table, steps[0].held, lens, new, fixed, steps[0].free_count)

        steps[0].block_table.copy_(torch.from_numpy(table))
        steps[0].held.copy_(torch.from_numpy(held))
        steps[0].free_count.fill_(len(free))
        graph = None
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                pair()
        want_table, want_held, left, at = table, held, len(free), list(past)
        for n in news:
            new.copy_(torch.tensor(n, dtype=torch.int32))
            lens.copy_(torch.tensor(at, dtype=torch.int32))
            want = step_ref.assign(want_table, want_held, at, n, free, left, page, tokens)
            if graph:
                graph.replay()
            else:
                stream.wait_stream(torch.cuda.current_stream())
                q4.q4_kv_assign(steps[1], steps[0].block_table, steps[0].held, lens, new, fixed, steps[0].free_count, stream=stream)
            torch.cuda.synchronize()
            assert np.array_equal(steps[1].block_table.cpu().numpy(), want["table"])
            assert steps[1].held.tolist() == want["held"].tolist() and steps[1].free_count.tolist() == [want["free"]]
            assert steps[1].slots.tolist()[: sum(n)] == want["slots"][: sum(n)]
            want_table, want_held, left, at = want["table"], want["held"], want["free"], [p + x for p, x in zip(at, n)]
            if graph:  # the captured step reads the first tables
                steps[0].block_table.copy_(steps[1].block_table)
                steps[0].held.copy_(steps[1].held)
                steps[0].free_count.copy_(steps[1].free_count)
            else:
                steps.reverse()

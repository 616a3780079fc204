"""q4_tree_accept and q4_kv_move against the same walk and copies on the host."""
import numpy as np
import pytest
import torch

import kv_ref
import step_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()


def drafts(new, rng, kind="random", right=0.7, vocab=50):
    """Parents, what the trunk chose behind each node, and drafts that are often that."""
    parents, choice, draft, first = [], [], [], 0
    for n in new:
        p = step_ref.tree(n, rng, kind)
        c = rng.integers(0, vocab, n)
        d = rng.integers(0, vocab, n)
        for i in range(1, n):
            if p[i] >= 0 and rng.random() < right:
                d[i] = c[p[i]]
        parents += p
        choice += list(c)
        draft += list(d)
        first += n
    return parents, choice, draft


def run(q4, new, ctx, parents, choice, draft, tokens, seqs_start=None, history=None):
    start = np.concatenate([[0], np.cumsum(new)]) if seqs_start is None else np.asarray(seqs_start)
    pad = tokens - len(choice)
    fill = lambda x: i32(list(x) + [3] * pad)  # noqa: E731
    table = torch.zeros(len(ctx), 1, dtype=torch.int32, device="cuda")
    batch = q4.KVBatch(table, i32(start), i32(ctx))
    h = None if history is None else i32(history)
    got = q4.q4_tree_accept(batch, fill(choice), fill(draft), parents=None if parents is None else fill(parents), history=h)
    host = None if history is None else history.copy()
    want = step_ref.accept(start, ctx, list(choice) + [3] * pad, list(draft) + [3] * pad, None if parents is None else list(parents) + [3] * pad,
                           tokens, host)
    torch.cuda.synchronize()
    accepted, following, path, lens = (x.tolist() for x in got)
    assert accepted == want[0] and following == want[1] and lens == want[3]
    assert [p for p, x in zip(path, want[2]) if x is not None] == [x for x in want[2] if x is not None]
    out = tuple(torch.full_like(x, -77) for x in got)
    assert q4.q4_tree_accept(batch, fill(choice), fill(draft), parents=None if parents is None else fill(parents), out=out) is out
    assert out[2].tolist() == [-77 if x is None else x for x in want[2]]
    assert all(torch.equal(out[i], got[i]) for i in (0, 1, 3))
    if history is not None:
        assert np.array_equal(h.cpu().numpy(), host)
    return got


@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("new", [[1], [2], [16], [64], [65, 0, 3], [200, 1, 64, 256], [257, 5, 700], [0, 0, 1]])
def test_accept(new, kind):
    q4 = lib()
    for seed, right in ((0, 0.7), (1, 1.0), (2, 0.0)):
        rng = np.random.default_rng(seed)
        parents, choice, draft = drafts(new, rng, kind, right, 3 if seed == 0 else 50)
        ctx = [n + int(rng.integers(0, 40)) for n in new]
        say("accept", new, kind, right)
        history = rng.integers(0, 9, (len(new), max(ctx) - 2 if max(ctx) > 4 else 3)).astype(np.int32)
        run(q4, new, ctx, parents, choice, draft, sum(new) + 2, history=history)
        run(q4, new, ctx, None, choice, draft, sum(new) + 2)


def test_accept_many_sequences():
    q4 = lib()
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 20, 777)]
    parents, choice, draft = drafts(new, rng)
    run(q4, new, [n + 3 for n in new], parents, choice, draft, sum(new))


def test_accept_odd_inputs():
    """Equal siblings (the lowest), several tokens without a parent (the first alone counts), parents that are none, a
    choice below 0 (a row with nothing allowed) which no draft matches, rows behind the call's."""
    q4 = lib()
    run(q4, [5], [9], [-1, 0, 0, 1, 2], [7, 8, 9, 1, 2], [4, 7, 7, 8, 9], 5)
    run(q4, [4], [4], [-1, -1, 1, 0], [5, 5, 5, 5], [5, 5, 5, 5], 4)
    run(q4, [4], [4], [3, 1, 7, -9], [5, 5, 5, 5], [5, 5, 5, 5], 4)
    run(q4, [4], [4], [-1, 0, 1, 2], [-1, -1, -1, -1], [-1, -1, -1, -1], 4)
    run(q4, [3, 4], [8, 9], [-1, 0, 1, -1, 0, 1, 2], [1] * 7, [1] * 7, 7, seqs_start=[0, 3, 9])  # the second's rows are not all there
    run(q4, [3], [2], [-1, 0, 1], [1] * 3, [1] * 3, 3, history=np.zeros((1, 5), np.int32))  # a past below 0
    with pytest.raises(ValueError):
        run(q4, [0], [0], [], [], [], 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layers,hk,dim,page,new,past", [(1, 8, 128, 16, [16], [170]), (3, 2, 64, 8, [30, 0, 64, 1], [5, 9, 0, 3]), (2, 1, 96, 24, [200, 100], [0, 77]),
                                                         (70, 1, 64, 8, [9, 12], [3, 4]), (2, 3, 33, 8, [40], [11]), (1, 40, 256, 32, [64], [100])])
def test_move(layers, hk, dim, page, new, past, dtype):
    """Paths over page borders, long ones, odd heads (element by element), more layers than a launch has; caches of which
    layers and sides lie beside each other in one tensor."""
    q4 = lib()
    rng = np.random.default_rng(dim)
    parents, choice, draft = drafts(new, rng, right=0.95)
    batch = kv_ref.Batch([(n, p + n) for n, p in zip(new, past)], page, seed=3, pad_rows=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    everything = torch.randn(batch.pages, layers, 2, hk, page, dim, device="cuda", generator=g).to(dtype)
    stack = q4.KVLayers([q4.KVCache(everything[:, i, 0], everything[:, i, 1]) for i in range(layers)])
    dev = batch.device(q4)
    accepted, _, path, _ = q4.q4_tree_accept(dev, i32(choice + [0]), i32(draft + [0]), parents=i32(parents + [0]))
    # the path the drafts make, whatever its length, and one of about half of the nodes
    some = [sorted({0} | set(rng.choice(n, n // 2, replace=False).tolist())) for n in new]
    made = i32([x for got, n in zip(some, new) for x in got + [-1] * (n - len(got))] + [0])
    for p, a in ((path, accepted), (made, i32([len(x) for x in some]))):
        before = everything.cpu().clone()
        q4.q4_kv_move(stack, dev, p, a)
        torch.cuda.synchronize()
        got, p, a = everything.cpu(), p.tolist(), a.tolist()
        for i in range(layers):
            for side in range(2):
                assert torch.equal(got[:, i, side], step_ref.move(before[:, i, side], batch.table, page, batch.pages, batch.start, batch.ctx, p, a)), (i, side)


def test_move_odd_paths():
    """Entries that are not above their index, not below the new tokens, or repeated; counts out of range; places
    without a page: nothing else is touched."""
    q4 = lib()
    page, hk, dim = 8, 2, 64
    batch = kv_ref.Batch([(12, 20), (6, 6), (10, 30)], page, seed=4)
    batch.table[2, 3] = -1  # the last places of the third have no page
    batch.table[1, 0] = batch.pages  # and none of the second's
    path = [0, 5, 5, 3, 2, 11, 99, 11, -1, 10, 9, 11] + [0, 2, 3, 4, 5, -1] + [0, 4, 5, 6, 9, 7, 8, 9, 9, 9]
    for accepted in ([12, 5, 10], [3, 6, 4], [99, 99, 99], [-5, 0, 1]):
        k, v = (torch.randn(batch.pages, hk, page, dim).half() for _ in range(2))
        kc, vc = k.cuda(), v.cuda()
        q4.q4_kv_move(q4.KVCache(kc, vc), batch.device(q4), i32(path), i32(accepted))
        torch.cuda.synchronize()
        for got, was in ((kc, k), (vc, v)):
            assert torch.equal(got.cpu(), step_ref.move(was, batch.table, page, batch.pages, batch.start, batch.ctx, path, accepted))


def test_move_far_pages():
    """Pages whose offsets pass 2^32 bytes."""
    q4 = lib()
    page, hk, dim = 64, 8, 128
    big = torch.zeros(36000, hk, page, dim, dtype=torch.float16, device="cuda")  # 4.7 GB
    vbig = torch.zeros(36000, hk, page, dim, dtype=torch.float16, device="cuda")
    table = i32([[35999, 35998]])
    big[35998, :, 3] = 2.0
    vbig[35998, :, 3] = 3.0
    batch = q4.KVBatch(table, i32([0, 8]), i32([68]))
    q4.q4_kv_move(q4.KVCache(big, vbig), batch, i32([0, 7] + [-1] * 6), i32([2]))
    torch.cuda.synchronize()
    assert bool((big[35999, :, 61] == 2.0).all()) and bool((vbig[35999, :, 61] == 3.0).all())
    assert float(big.sum()) == 2 * 2.0 * hk * dim

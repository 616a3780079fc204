"""q4_attention_tree against attention in 64 bits over the keys that each row's mask names."""
import math

import numpy as np
import pytest
import torch

import attention_cuts
import kv_ref
import step_ref
import tree_cuts
from gpu_util import lib, say

pytestmark = pytest.mark.gpu
BOTH = [torch.float16, torch.bfloat16]


def setup(lens, page, hq, hk, dim, dtype, words=1, seed=0, pad_rows=0, columns=0, kind="random"):
    batch = kv_ref.Batch(lens, page, seed=seed, pad_rows=pad_rows, columns=columns)
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(batch.pages, hk, page, dim, generator=g).to(dtype) for _ in range(2))
    q = (1.5 * torch.randn(batch.tokens, hq, dim, generator=g)).to(dtype)
    rng = np.random.default_rng(seed)
    mask = step_ref.mask_rows([step_ref.tree(n, rng, kind) for n in batch.new], words)
    mask = torch.cat([mask, torch.full((batch.tokens - mask.shape[0], words), -1, dtype=torch.int64)])
    return batch, q, k, v, mask


def check(q4, batch, q, k, v, mask, window=0, hint=None, scale=None, exact=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    exact = exact or step_ref.TreeExact(q, k, v, batch, mask, scale, window)
    n = int(batch.start[-1])
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    q4.q4_attention_tree(q4.KVCache(k.cuda(), v.cuda()), batch.device(q4, hint), q.cuda(), mask.cuda(), scale=scale, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    err = (out[:n].double().cpu() - exact.out[:n]).abs()
    assert bool((err <= exact.bound[:n]).all()), float((err / exact.bound[:n]).max())
    some = torch.isfinite(exact.lse[:n])
    assert torch.equal(lse[:n].cpu()[~some], torch.full((int((~some).sum()),), -math.inf)) and bool((out[:n].cpu()[~some] == 0).all())
    assert bool(((lse[:n].double().cpu() - exact.lse[:n]).abs()[some] <= exact.lse_bound[:n][some]).all())
    assert bool((out[n:] == 5.0).all()) and bool((lse[n:] == 5.0).all())
    return out, exact


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("case", tree_cuts.cases(), ids=repr)
def test_every_kernel(case, dtype):
    """Items of 16 to 128 rows, whole and cut, every head_dim, with and without a window (a CPU test checks that these calls are cut
    like that)."""
    q4 = lib()
    say("tree", case, dtype)
    batch = case.batch(3)
    words = -(-max(batch.new) // 64)
    _, q, k, v, mask = setup(case.lens, case.page, case.hq, case.hk, case.dim, dtype, words, 3, case.pad, case.columns)
    dev = q4.KVBatch(torch.from_numpy(batch.table).cuda(), torch.from_numpy(batch.start).cuda(), torch.tensor(batch.ctx, dtype=torch.int32, device="cuda"),
                     max_query_len=case.max_query, max_context_len=case.max_context)
    exact = step_ref.TreeExact(q, k, v, batch, mask, case.dim ** -0.5, case.window)
    n = int(batch.start[-1])
    cache = q4.KVCache(k.cuda(), v.cuda())
    out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
    q4.q4_attention_tree(cache, dev, q.cuda(), mask.cuda(), window=case.window, out=out)
    torch.cuda.synchronize()
    err = (out[:n].double().cpu() - exact.out[:n]).abs()
    assert bool((err <= exact.bound[:n]).all()), float((err / exact.bound[:n]).max())
    assert bool((out[n:] == 5.0).all())


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("past", [0, 1, 31, 32, 33, 63, 64, 65, 127, 500, 2047])
@pytest.mark.parametrize("n", [1, 2, 17, 33, 64])
def test_borders(n, past, dtype):
    """Trees that begin and end at every place of a step and a tile, of one token to 64, few and many rows."""
    q4 = lib()
    for hq in (2, 16):
        check(q4, *setup([(n, past + n)], 16, hq, 2, 64, dtype, 1, n + past))


@pytest.mark.parametrize("words", [1, 2, 3, 4])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
def test_long_masks(words, kind):
    """Trees over several words, and longer than the mask (what has no bit is not seen, not even by itself)."""
    q4 = lib()
    lens = [(200, 300), (64, 64), (65, 70), (0, 9), (1, 300), (130, 1000)]
    for hq in (2, 8):
        check(q4, *setup(lens, 24, hq, 2, 128, torch.float16, words, 5, 2, kind=kind))


@pytest.mark.parametrize("dtype", BOTH)
def test_any_bits(dtype):
    """Masks that are no trees: nothing at all (with and without a cache behind it), everything, later tokens, not the
    row itself, bits behind the new tokens."""
    q4 = lib()
    lens = [(9, 9), (40, 140), (70, 70), (3, 500), (5, 5)]
    for hq, words in ((2, 2), (8, 2), (16, 3)):
        batch, q, k, v, _ = setup(lens, 16, hq, 2, 64, dtype, words, 6)
        g = torch.Generator().manual_seed(9)
        for mask in (torch.zeros(batch.tokens, words, dtype=torch.int64), torch.full((batch.tokens, words), -1, dtype=torch.int64),
                     torch.randint(-2 ** 63, 2 ** 63 - 1, (batch.tokens, words), generator=g),
                     torch.randint(0, 2, (batch.tokens, words), generator=g) << 62):
            for window in (0, 1, 30):
                check(q4, batch, q, k, v, mask, window)


@pytest.mark.parametrize("window", [1, 2, 7, 64, 100, 700, 2 ** 40])
def test_windows(window):
    """Windows from the row's own token to longer than the context."""
    q4 = lib()
    lens = [(30, 900), (1, 900), (64, 64), (12, 77), (60, 3000)]
    for hq in (2, 4, 16):
        batch, q, k, v, mask = setup(lens, 32, hq, 2, 128, torch.bfloat16, 1, 8)
        check(q4, batch, q, k, v, mask, window)


def test_a_chain_is_causal():
    """With the mask of a chain, with and without a window, what attention over causal rows is (which the bounds are
    those of, too)."""
    q4 = lib()
    for lens, hq in (([(5, 700), (1, 33)], 4), ([(60, 900), (64, 64)], 8)):
        batch, q, k, v, mask = setup(lens, 16, hq, 2, 128, torch.float16, 1, 2, kind="chain")
        check(q4, batch, q, k, v, mask, exact=attention_cuts.Exact(q, k, v, batch, 128 ** -0.5, 0))
        exact = attention_cuts.Exact(q, k, v, batch, 128 ** -0.5, 50)
        # a window reaches into the chain: its first tokens are out of sight of the last
        inside = step_ref.mask_rows([step_ref.tree(n, None, "chain") for n in batch.new], 1)
        at = 0
        for n in batch.new:
            for i in range(n):
                for j in range(max(0, i - 49)):
                    inside[at + i, 0] &= ~(1 << j)
            at += n
        check(q4, batch, q, k, v, inside, 50, exact=exact)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("hq", [2, 32])
def test_values_that_are_not_finite(hq, dtype):
    """NaN and infinities in tokens that a row does not see (other branches, slots behind the context, pages it does not
    have) leave it as it is; in one that it sees they reach it and no other."""
    q4 = lib()
    lens = [(30, 120), (64, 100), (1, 50)]
    batch, q, k, v, mask = setup(lens, 16, hq, 2, 64, dtype, 1, 11)
    want, _ = check(q4, batch, q, k, v, mask)
    places = {b: {p: (pg, s) for p, pg, s in batch.places(b)} for b in range(3)}
    used = {x for b in places for x in places[b].values()}
    k2, v2 = k.clone(), v.clone()
    for pg in range(batch.pages):
        for s in range(16):
            if (pg, s) not in used:
                k2[pg, :, s] = float("nan")
                v2[pg, :, s] = float("inf")
    plain = v2
    for node in (7, 0, 3, 63):  # of the second sequence: a leaf, the root, others
        pg, s = places[1][36 + node]
        v2 = plain.clone()
        v2[pg, :, s, 3] = float("inf")
        v2[pg, :, s, 4] = float("nan")
        out = q4.q4_attention_tree(q4.KVCache(k2.cuda(), v2.cuda()), batch.device(q4), q.cuda(), mask.cuda())
        sees = torch.tensor([r >= 30 and r < 94 and bool((int(mask[r, 0]) >> node) & 1) for r in range(batch.tokens)])
        assert int(sees.sum()) >= (64 if node == 0 else 1)
        assert torch.equal(out[~sees.cuda()], want[~sees.cuda()])
        hit = out[sees.cuda()]
        assert bool((hit[..., 3] == math.inf).all()) and bool(torch.isnan(hit[..., 4]).all())
        clean = torch.tensor([e not in (3, 4) for e in range(64)])
        assert torch.equal(hit[..., clean], want[sees.cuda()][..., clean])
        k3 = k.clone()
        k3[pg, :, s] = float("nan")
        out = q4.q4_attention_tree(q4.KVCache(k3.cuda(), v.cuda()), batch.device(q4), q.cuda(), mask.cuda())
        assert torch.equal(out[~sees.cuda()], want[~sees.cuda()]) and bool(torch.isnan(out[sees.cuda()]).all())


def test_places_that_are_missing():
    """Pages that are not there, tables that are too short, contexts shorter than their new tokens."""
    q4 = lib()
    batch, q, k, v, mask = setup([(20, 200), (40, 90), (30, 31)], 16, 8, 2, 128, torch.float16, 1, 12)
    batch.table[0, 3] = -1
    batch.table[0, 12] = batch.pages  # of new tokens
    batch.table[1, :] = -1
    check(q4, batch, q, k, v, mask)
    batch.ctx[2] = 25  # places below 0: the first five
    check(q4, batch, q, k, v, mask)
    batch.table = batch.table[:, :2].copy()
    check(q4, batch, q, k, v, mask)


def test_strided_heads_and_groups():
    """Queries that are a part of packed rows, a cache with slots before heads, groups that no item's rows divide."""
    q4 = lib()
    for hq, hk in ((20, 1), (33, 1), (7, 7), (12, 4)):
        batch, q, k, v, mask = setup([(9, 100), (1, 40), (50, 77)], 16, hq, hk, 128, torch.bfloat16, 1, hq)
        want, exact = check(q4, batch, q, k, v, mask)
        wide = torch.zeros(batch.tokens, hq + 3, 128, dtype=torch.bfloat16, device="cuda")
        wide[:, 1 : hq + 1] = q.cuda()
        kt, vt = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (k, v))
        got = q4.q4_attention_tree(q4.KVCache(kt, vt), batch.device(q4), wide[:, 1 : hq + 1], mask.cuda())
        assert torch.equal(got, want)


def test_two_streams_and_a_workspace():
    """Calls cut into parts on two streams at once, each with a workspace of its own."""
    q4 = lib()
    jobs = []
    for seed, lens in enumerate(([(8, 9000), (3, 200)], [(64, 6000)])):
        batch, q, k, v, mask = setup(lens, 32, 4, 2, 128, torch.bfloat16, 1, seed)
        cache, dev, dq = q4.KVCache(k.cuda(), v.cuda()), batch.device(q4), q.cuda()
        need = q4.attention_tree_workspace_bytes(cache, dev, 4, batch.tokens)
        assert need > 0
        want, _ = check(q4, batch, q, k, v, mask)
        jobs.append((cache, dev, dq, mask.cuda(), want, torch.cuda.Stream(), torch.empty(need, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (cache, dev, dq, m, _, stream, ws) in enumerate(jobs):
            got[i].append(q4.q4_attention_tree(cache, dev, dq, m, workspace=ws, stream=stream))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for out in got[i]:
            assert torch.equal(out, job[4])


@pytest.mark.parametrize("dtype", BOTH)
def test_captured_with_new_trees(dtype):
    """A graph of a call cut into parts and of one taken whole, replayed with other lengths, trees and tables in the same
    tensors, eager calls in between; both graphs use one workspace, one after the other."""
    q4 = lib()
    page, hq, hk, dim, tokens = 32, 8, 2, 128, 40
    steps = [setup(lens, page, hq, hk, dim, dtype, 1, seed, tokens - sum(n for n, _ in lens), 300)
             for seed, lens in enumerate(([(16, 9000), (20, 300)], [(1, 1), (0, 4000)], [(40, 40), (0, 0)], [(3, 6001), (33, 8999)]))]
    pages = max(s[0].pages for s in steps)
    k, v = (torch.zeros(pages, hk, page, dim, dtype=dtype, device="cuda") for _ in range(2))
    cache, q = q4.KVCache(k, v), torch.zeros(tokens, hq, dim, dtype=dtype, device="cuda")
    mask = torch.zeros(tokens, 1, dtype=torch.int64, device="cuda")
    table, start, ctx = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((2, 300), (3,), (2,)))
    out = torch.zeros(tokens, hq, dim, dtype=dtype, device="cuda")
    batches = [q4.KVBatch(table, start, ctx, max_query_len=40, max_context_len=n) for n in (9600, 40)]
    need = [q4.attention_tree_workspace_bytes(cache, b, hq, tokens) for b in batches]
    assert need[0] > 0
    ws = torch.empty(max(need), dtype=torch.uint8, device="cuda")
    graphs = []
    for b in batches:
        q4.q4_attention_tree(cache, b, q, mask, out=out, workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            q4.q4_attention_tree(cache, b, q, mask, out=out, workspace=ws)
    for batch, hq_, hk_, hv_, hm in steps * 2:
        k[: batch.pages].copy_(hk_)
        v[: batch.pages].copy_(hv_)
        q.copy_(hq_)
        mask.copy_(hm)
        table.copy_(torch.from_numpy(batch.table))
        start.copy_(torch.from_numpy(batch.start))
        ctx.copy_(torch.tensor(batch.ctx, dtype=torch.int32))
        n = int(batch.start[-1])
        exact = step_ref.TreeExact(hq_, hk_, hv_, batch, hm, dim ** -0.5, 0)
        for graph, b in zip(graphs, batches):
            out.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            first = out.clone()
            err = (first[:n].double().cpu() - exact.out[:n]).abs()
            assert bool((err <= exact.bound[:n]).all()) and bool((first[n:] == 5.0).all())
            assert torch.equal(q4.q4_attention_tree(cache, b, q, mask, workspace=ws)[:n], first[:n])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)


@pytest.mark.parametrize("heads", [(8, 8), (40, 8)])
def test_far_pages(heads):
    """A cache of which some pages lie behind 2^32 bytes, read by items of few rows and by tiles, and written by an append
    with norms: the same as in a small cache."""
    q4 = lib()
    hq, hk = heads
    page, dim, pages = 64, 128, 36000
    batch, q, k, v, mask = setup([(16, 700), (30, 1500)], page, hq, hk, dim, torch.bfloat16, 1, 4)
    far = pages - batch.pages
    caches = []
    for count, first in ((batch.pages, 0), (pages, far)):
        ck, cv = (torch.zeros(count, hk, page, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ck[first:].copy_(k)
        cv[first:].copy_(v)
        table = torch.from_numpy(batch.table).cuda() + first
        dev = q4.KVBatch(table, torch.from_numpy(batch.start).cuda(), torch.tensor(batch.ctx, dtype=torch.int32, device="cuda"))
        x = q[:, :hk].cuda()
        q4.q4_kv_append_norm(q4.KVCache(ck, cv), dev, x, 2 * x, inv_freq=q4.rope_frequencies(dim)[0])
        caches.append((ck[first:], cv[first:], q4.q4_attention_tree(q4.KVCache(ck, cv), dev, q.cuda(), mask.cuda())))
    assert not torch.equal(caches[0][0].cpu(), k)
    for a, b in zip(*caches):
        assert torch.equal(a, b)

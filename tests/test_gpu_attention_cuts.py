"""Every attention kernel, whole and cut (tests/attention_cuts.py; that the calls are cut as they say is tested on the
CPU), against the same in 64 bits: masks, windows, slots without a token, log-sum-exp, values and keys that are not
finite, block tables and caches of any strides."""
import math

import pytest
import torch

import kv_ref
from attention_cuts import Exact, cases
from gpu_util import lib, say

pytestmark = pytest.mark.gpu

CASES = cases()


def data(case, dtype, seed):
    """Queries, and keys and values of different strides whose slots without a token hold NaN and infinities."""
    batch = case.batch(seed)
    g = torch.Generator().manual_seed(seed)
    order = ((0, 1, 2, 3), (0, 2, 1, 3))
    k, v = (torch.randn([(batch.pages, case.hk, batch.page, case.dim)[i] for i in o], generator=g).to(dtype).permute(o)
            for o in (order[seed % 2], order[(seed + 1) % 2]))
    used = torch.zeros(batch.pages, batch.page, dtype=torch.bool)
    for b in range(len(batch.new)):
        for _, page, slot in batch.places(b):
            used[page, slot] = True
    junk = torch.tensor([math.nan, math.inf, -math.inf])
    for x in (k, v):
        holes = ~used[:, None, :, None].expand(x.shape)
        x[holes] = junk[torch.randint(0, 3, (int(holes.sum()),), generator=g)].to(dtype)
    q = torch.randn(batch.tokens, case.hq, case.dim, generator=g).to(dtype)
    return batch, q, k, v


def gpu_batch(q4, case, batch):
    """The batch, its block table's rows further apart than they are wide, with page numbers of nobody between."""
    wide = torch.full((len(batch.new), batch.table.shape[1] + 3), 7777777, dtype=torch.int32, device="cuda")
    wide[:, : batch.table.shape[1]] = torch.from_numpy(batch.table)
    return q4.KVBatch(wide[:, : batch.table.shape[1]], torch.from_numpy(batch.start).cuda(),
                      torch.tensor(batch.ctx, dtype=torch.int32, device="cuda"), max_query_len=case.max_query,
                      max_context_len=case.max_context)


def on_gpu(x):
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def run(q4, case, batch, q, k, v):
    cache, dev = q4.KVCache(on_gpu(k), on_gpu(v)), gpu_batch(q4, case, batch)
    assert (q4.attention_workspace_bytes(cache, dev, case.hq, batch.tokens, case.window) == 0) == case.whole
    out, lse = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda"), torch.full(q.shape[:2], 5.0, device="cuda")
    q4.q4_attention_paged(cache, dev, q.cuda(), window=case.window, out=out, lse=lse)
    torch.cuda.synchronize()
    n = int(batch.start[-1])
    assert bool((out[n:] == 5.0).all()) and bool((lse[n:] == 5.0).all())  # rows behind the last sequence
    return out[:n].cpu(), lse[:n].cpu()


def same_bits(a, b):
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("index", range(len(CASES)), ids=[repr(c) for c in CASES])
def test_every_kernel(index, dtype):
    q4, case = lib(), CASES[index]
    say("attention", case, dtype)
    batch, q, k, v = data(case, dtype, index)
    n = int(batch.start[-1])
    exact = Exact(q, k, v, batch, case.dim ** -0.5, case.window)
    out, lse = run(q4, case, batch, q, k, v)
    want, bound = exact.out[:n], exact.bound[:n]
    assert bool(((out.double() - want).abs() <= bound).all())
    none = torch.isinf(exact.lse[:n])
    assert bool((lse[none] == -math.inf).all()) and bool((out[none] == 0).all())
    assert bool(((lse.double() - exact.lse[:n]).abs() <= exact.lse_bound[:n])[~none].all())

    # Values that are not finite, one of them in the context and two in the new tokens of each sequence: a row that
    # sees one of them with a weight w has w times it in its sum, the others and all else are as before.
    bad_v, want, touched = v.clone(), want.clone(), torch.zeros(out.shape, dtype=torch.bool)
    for b in exact.weights:
        first = batch.ctx[b] - batch.new[b]
        rows = slice(int(batch.start[b]), int(batch.start[b + 1]))
        places = batch.places(b)
        of = {p: i for i, (p, _, _) in enumerate(places)}
        for p, column, bad in ((3, 7, math.inf), (first, 9, math.nan), (first + batch.new[b] // 2, 11, -math.inf),
                               (first, 11, math.inf), (batch.ctx[b] - 1, 13, math.inf)):
            if p not in of or (column == 11 and bad > 0 and batch.new[b] < 2):  # (one new token: 11 is taken)
                continue
            _, page, slot = places[of[p]]
            bad_v[page, :, slot, column] = bad
            sees = exact.seen(b, torch.tensor([p]))[:, 0]
            w = exact.weights[b][:, :, of[p]].transpose(0, 1)  # rows, heads
            add = torch.where(sees[:, None], w * bad, torch.zeros_like(w))
            want[rows, :, column] += add
            touched[rows, :, column] |= sees[:, None]
    got, got_lse = run(q4, case, batch, q, k, bad_v)
    assert same_bits(got[~touched], out[~touched]) and same_bits(got_lse, lse)
    expect, have = want[touched], got[touched].double()
    assert not bool(torch.isfinite(expect).any())
    nan = torch.isnan(expect)
    assert bool((torch.isnan(have) == nan).all()) and bool((have == expect)[~nan].all())

    # Keys that are not finite.  NaN, and an infinity that a query turns into a score of +infinity: the rows that see
    # the key are NaN, the others as before.
    q[:, :, 5] = 1.0
    out, lse = run(q4, case, batch, q, k, v)
    rows_nan = torch.zeros(n, dtype=torch.bool)
    bad_k, low_k, far_k = k.clone(), k.clone(), k.clone()
    for b in exact.weights:
        first = batch.ctx[b] - batch.new[b]
        p = first + batch.new[b] // 2
        if p < 0:
            continue
        _, page, slot = batch.places(b)[p]
        bad_k[page, :, slot, 5] = math.nan if b % 2 else math.inf
        low_k[page, :, slot, 5], far_k[page, :, slot, 5] = -math.inf, -30000.0
        rows_nan[int(batch.start[b]) : int(batch.start[b + 1])] = exact.seen(b, torch.tensor([p]))[:, 0]
    got, got_lse = run(q4, case, batch, q, bad_k, v)
    assert bool(torch.isnan(got[rows_nan]).all()) and bool(torch.isnan(got_lse[rows_nan]).all())
    assert same_bits(got[~rows_nan], out[~rows_nan]) and same_bits(got_lse[~rows_nan], lse[~rows_nan])
    # a score of -infinity: a weight of 0, as of a score of -30000 / sqrt(dim), less than -1800 (2^-2600 of the others);
    # of a row that sees no other key the sum of weights is 0 in the one case, and 1 in the other
    got, got_lse = run(q4, case, batch, q, low_k, v)
    far, far_lse = run(q4, case, batch, q, far_k, v)
    other = ~(torch.isinf(got_lse) & (far_lse < -1000))
    assert same_bits(got[other], far[other]) and same_bits(got_lse[other], far_lse[other])
    assert bool((got[~other] == 0).all())

"""Uses of the cache operators that their documentation allows: any number of query heads for a kv head, broadcast
inputs, windows longer than any context, two streams at once, graphs of prompt chunks."""
import pytest
import torch

import kv_ref
from attention_cuts import Exact
from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def setup(lens, page, hq, hk, dim, dtype, seed=0, pad_rows=0, columns=0):
    batch = kv_ref.Batch(lens, page, seed=seed, pad_rows=pad_rows, columns=columns)
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(batch.pages, hk, page, dim, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(batch.tokens, hq, dim, generator=g).to(dtype)
    return batch, q, k, v


def close(out, exact, rows):
    assert bool(((out[:rows].double().cpu() - exact.out[:rows]).abs() <= exact.bound[:rows]).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hk,dim", [(20, 1, 64), (33, 1, 128), (66, 2, 96), (130, 1, 64), (512, 2, 128), (71, 71, 64), (96, 3, 256)])
def test_any_number_of_query_heads(hq, hk, dim, dtype):
    """Groups of 1 to 256 query heads, not of a size that divides an item's rows: one token's heads in several items,
    an item of several tokens' heads."""
    q4 = lib()
    say("heads", hq, hk, dim, dtype)
    lens = [(1, 100), (1, 1), (0, 5), (2, 300), (1, 65), (5, 64)]
    batch, q, k, v = setup(lens, 16, hq, hk, dim, dtype, pad_rows=2)
    n = int(batch.start[-1])
    exact = Exact(q, k, v, batch, dim ** -0.5, 0)
    cache = q4.KVCache(k.cuda(), v.cuda())
    for hint in (None, 5, 1):
        out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
        q4.q4_attention_paged(cache, batch.device(q4, hint), q.cuda(), out=out)
        close(out, exact, n)
        assert bool((out[n:] == 5.0).all())


def test_broadcast_inputs():
    """Queries that are one row for all tokens, keys and values that are one head for all kv heads, a window longer
    than 31 bits: as of tensors that hold them all."""
    q4 = lib()
    batch, q, k, v = setup([(4, 30), (30, 90), (1, 700)], 16, 8, 2, 64, torch.float16)
    cache, dev = q4.KVCache(k.cuda(), v.cuda()), batch.device(q4)
    one = q[:1].cuda().expand(batch.tokens, 8, 64)
    assert one.stride(0) == 0
    want = q4.q4_attention_paged(cache, dev, one.contiguous())
    assert torch.equal(q4.q4_attention_paged(cache, dev, one), want)
    assert torch.equal(q4.q4_attention_paged(cache, dev, one, window=2 ** 40), want)
    head = q[:, :1].cuda().expand(batch.tokens, 2, 64)
    assert head.stride(1) == 0
    freq, _ = q4.rope_frequencies(64)
    pos = torch.arange(batch.tokens, dtype=torch.int32, device="cuda")
    assert torch.equal(q4.q4_rope(head, pos, freq), q4.q4_rope(head.contiguous(), pos, freq))
    caches = []
    for x in (head, head.contiguous()):
        c = q4.KVCache(torch.zeros_like(cache.k), torch.zeros_like(cache.v))
        q4.q4_kv_append(c, dev, x, x, inv_freq=freq)
        caches.append(c)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


def test_two_streams_at_once():
    """Decode and prompt calls on two streams, in turn and over and over, each with parts in a workspace of its own."""
    q4 = lib()
    jobs = []
    for seed, lens in enumerate(([(1, 9000), (1, 200)], [(64, 4000)])):
        batch, q, k, v = setup(lens, 32, 4, 2, 128, torch.bfloat16, seed)
        cache, dev, dq = q4.KVCache(k.cuda(), v.cuda()), batch.device(q4), q.cuda()
        assert q4.attention_workspace_bytes(cache, dev, 4, batch.tokens) > 0
        want = q4.q4_attention_paged(cache, dev, dq)
        close(want, Exact(q, k, v, batch, 128 ** -0.5, 0), batch.tokens)
        jobs.append((cache, dev, dq, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (cache, dev, dq, _, stream) in enumerate(jobs):
            got[i].append(q4.q4_attention_paged(cache, dev, dq, stream=stream))
    torch.cuda.synchronize()
    for i, job in enumerate(jobs):
        for out in got[i]:
            assert torch.equal(out, job[3])


@pytest.mark.parametrize("most,context", [(150, 300), (150, 60000), (6, 60000)])
def test_captured_chunks(most, context):
    """A graph of the append and attention of a prompt's chunk, whole and in parts, replayed with other lengths, pages
    and tokens in the same tensors, eager work of other sizes in between: every replay as the eager call."""
    q4 = lib()
    page, hq, hk, dim, rows = 16, 4, 2, 64, 200
    columns = -(-max(context, 1000) // page)
    steps = [[(150, 150), (1, 700)], [(6, 40), (3, 800)], [(0, 0), (140, 900)], [(5, 5), (6, 6)]]
    if most < 150:
        steps = [[(min(n, most), c) for n, c in lens] for lens in steps]
    batches = [kv_ref.Batch(lens, page, spare=150, seed=i, columns=columns) for i, lens in enumerate(steps)]
    pages = max(b.pages for b in batches)
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(pages, hk, page, dim, generator=g).half().cuda() for _ in range(2))
    cache = q4.KVCache(kc, vc)
    table, start, ctx = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, columns), (3,), (2,)))
    batch = q4.KVBatch(table, start, ctx, max_query_len=most, max_context_len=context)
    packed = torch.zeros(rows, (hq + 2 * hk) * dim, device="cuda")
    q, k, v = packed.view(rows, -1, dim).split([hq, hk, hk], 1)
    freq, _ = q4.rope_frequencies(dim)
    out, lse = torch.zeros(rows, hq, dim, dtype=torch.float16, device="cuda"), torch.zeros(rows, hq, device="cuda")
    assert (q4.attention_workspace_bytes(cache, batch, hq, rows) > 0) == (context > 1000)

    def step(o, l):
        turned = q4.q4_kv_append(cache, batch, k, v, q=q, inv_freq=freq)
        q4.q4_attention_paged(cache, batch, turned, out=o, lse=l)

    def load(i):
        b = batches[i % len(batches)]
        table.copy_(torch.from_numpy(b.table))
        start.copy_(torch.from_numpy(b.start))
        ctx.copy_(torch.tensor(b.ctx, dtype=torch.int32))
        packed.copy_(torch.randn(packed.shape, generator=g))

    load(0)
    step(out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, lse)
    for i in range(8):
        load(i)
        for x in (out, lse):
            x.fill_(3.0)
        kc0, vc0 = kc.clone(), vc.clone()
        graph.replay()
        torch.cuda.synchronize()
        got_k, got_v = kc.clone(), vc.clone()
        kc.copy_(kc0)
        vc.copy_(vc0)
        want, want_lse = torch.full_like(out, 3.0), torch.full_like(lse, 3.0)
        step(want, want_lse)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i
        assert torch.equal(kc, got_k) and torch.equal(vc, got_v), i
        q4.q4_attention_paged(cache, batch, torch.zeros(17, 8, dim, dtype=torch.float16, device="cuda"))  # other sizes

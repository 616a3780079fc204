"""Attention of new tokens over a paged cache, against the same in 64 bits, row by row."""
import math

import numpy as np
import pytest
import torch

import kv_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def make(batch, hq, hk, dim, dtype, seed=0, slots_first=False, spread=2.0):
    """Queries and a cache whose slots without a token hold NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    shape = (batch.pages, batch.page, hk, dim) if slots_first else (batch.pages, hk, batch.page, dim)
    order = (0, 2, 1, 3) if slots_first else (0, 1, 2, 3)
    k, v = (torch.randn(shape, generator=g).to(dtype).permute(order) for _ in range(2))
    used = torch.zeros(batch.pages, batch.page, dtype=torch.bool)
    for b in range(len(batch.new)):
        for _, page, slot in batch.places(b):
            used[page, slot] = True
    junk = torch.tensor([math.nan, math.inf, -math.inf])
    for x in (k, v):
        holes = ~used[:, None, :, None].expand(x.shape)
        x[holes] = junk[torch.randint(0, 3, (int(holes.sum()),), generator=g)].to(dtype)
    q = (torch.randn(batch.tokens, hq, dim, generator=g) * spread).to(dtype)
    return q, k, v


def on_gpu(x):
    """The same strides on the device."""
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return y.copy_(x)


def check(q4, batch, q, k, v, window=0, scale=None, max_query_len=None, what=""):
    scale = scale or q.shape[2] ** -0.5
    want, want_lse, bound, lse_bound = kv_ref.attention(q, k, v, batch, scale, window)
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    q4.q4_attention_paged(q4.KVCache(on_gpu(k), on_gpu(v)), batch.device(q4, max_query_len), q.cuda(), scale=scale,
                          window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    n = int(batch.start[-1])
    got, got_lse = out.double().cpu(), lse.double().cpu()
    bad = ~((got - want).abs() <= bound)[:n]
    assert not bad.any(), "%s: %d outside, first at %s, worst %g of the bound" % (
        what, int(bad.sum()), bad.nonzero()[0].tolist(), float(((got - want).abs() / bound)[:n].nan_to_num(1e9).max()))
    empty = torch.isinf(want_lse)
    assert bool((got_lse[:n][empty[:n]] == -math.inf).all())
    off = (got_lse - want_lse)[:n][~empty[:n]].abs()
    # the weights it sums are rounded (half a step each), and their exponents are off by the scores' error
    assert off.numel() == 0 or bool((off <= lse_bound[:n][~empty[:n]]).all())
    assert bool((out[n:] == 5.0).all()) and bool((lse[n:] == 5.0).all())  # rows behind the last sequence
    return out


CASES = [
    # new tokens and context of each sequence, page, query heads, kv heads, head, window
    ([(1, 1)], 16, 1, 1, 64, 0),
    ([(1, 33)], 8, 4, 4, 128, 0),
    ([(1, 515)], 16, 40, 40, 128, 0),
    ([(1, 700), (1, 1), (1, 64), (1, 65), (1, 2000)], 64, 32, 8, 128, 0),
    ([(1, c) for c in range(1, 140)], 24, 5, 1, 64, 0),
    ([(4, 600), (4, 4), (4, 100)], 32, 8, 8, 128, 0),
    ([(16, 300), (3, 3), (0, 50), (16, 16), (0, 0), (7, 999)], 16, 12, 4, 96, 0),
    ([(17, 170)], 16, 10, 2, 256, 0),
    ([(169, 169)], 16, 4, 4, 128, 0),
    ([(130, 500), (64, 64), (1, 300)], 128, 8, 1, 64, 0),
    ([(65, 700), (200, 201)], 40, 6, 2, 128, 0),
    ([(5, 2)], 8, 2, 2, 64, 0),  # more new tokens than context: the first three rows see nothing
    ([(1, 900), (20, 900), (100, 130)], 16, 8, 2, 64, 1),
    ([(1, 900), (20, 900), (100, 130)], 24, 8, 2, 128, 100),
    ([(300, 1000)], 32, 4, 1, 96, 257),
    ([(64, 300)], 64, 2, 1, 256, 33),
    ([(5, 300), (6, 77), (1, 1)], 16, 10, 2, 64, 0),     # 17 .. 32 rows of a kv head
    ([(5, 300), (6, 77), (1, 1)], 24, 10, 2, 96, 50),
    ([(5, 2000), (6, 77), (1, 1)], 16, 10, 2, 128, 0),
    ([(5, 300), (6, 1500), (1, 1)], 8, 10, 2, 256, 0),
    ([(64, 4000)], 32, 4, 2, 128, 0),                    # few items of many rows: cut
    ([(40, 5000), (130, 2500)], 64, 4, 1, 64, 3001),
    ([(33, 3500)], 16, 2, 1, 256, 0),
    ([(1, 6000)], 16, 2, 1, 256, 0),
    ([(1, 20000), (1, 3)], 128, 8, 1, 128, 0),
    ([(1, 9000)] + [(0, 50)] * 70 + [(1, 100)] * 3, 64, 4, 1, 96, 0),  # more than 64 sequences, most without new tokens
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype):
    q4 = lib()
    lens, page, hq, hk, dim, window = CASES[case]
    say("attention", case, lens[:6], page, hq, hk, dim, window, dtype)
    batch = kv_ref.Batch(lens, page, seed=case, pad_rows=2, columns=0 if case % 2 else 70)
    q, k, v = make(batch, hq, hk, dim, dtype, seed=case, slots_first=case % 3 == 0)
    check(q4, batch, q, k, v, window, what=str(case))


@pytest.mark.parametrize("hint", [1, 7, 100000])
def test_hints_do_not_change_what_is_computed(hint):
    q4 = lib()
    batch = kv_ref.Batch([(40, 300), (1, 77)], 16, seed=2)
    q, k, v = make(batch, 8, 2, 128, torch.float16)
    check(q4, batch, q, k, v, max_query_len=hint)


@pytest.mark.parametrize("hint", [1, 100, 10 ** 6])
def test_a_wrong_longest_context_does_not_change_what_is_computed(hint):
    q4 = lib()
    for lens in ([(1, 3000), (1, 5)], [(40, 3000), (3, 70)]):
        batch = kv_ref.Batch(lens, 16, seed=2)
        q, k, v = make(batch, 4, 2, 64, torch.bfloat16)
        want, _, bound, _ = kv_ref.attention(q, k, v, batch, 0.125, 0)
        dev = q4.KVBatch(*batch.device(q4)._keep, max_context_len=hint)
        out = q4.q4_attention_paged(q4.KVCache(on_gpu(k), on_gpu(v)), dev, q.cuda(), scale=0.125)
        assert bool(((out.double().cpu() - want).abs() <= bound).all())


def test_keys_and_values_of_one_tensor_and_queries_in_place():
    """Keys and values side by side in one tensor, queries turned in their place in packed rows."""
    q4 = lib()
    page, hq, hk, dim, n = 16, 4, 2, 64, 21
    g = torch.Generator().manual_seed(3)
    both = torch.zeros(5, 2, hk, page, dim, dtype=torch.float16, device="cuda")
    cache = q4.KVCache(both[:, 0], both[:, 1])
    plain = q4.KVCache(torch.zeros(5, hk, page, dim, dtype=torch.float16, device="cuda"),
                       torch.zeros(5, hk, page, dim, dtype=torch.float16, device="cuda"))
    packed = torch.randn(n, (hq + 2 * hk) * dim, generator=g).half().cuda()
    q, k, v = packed.view(n, -1, dim).split([hq, hk, hk], 1)
    kv = packed[:, hq * dim:].clone()
    batch = q4.KVBatch(torch.tensor([[3, 1]], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"))
    freq, _ = q4.rope_frequencies(dim)
    want = q4.q4_attention_paged(plain, batch, q4.q4_kv_append(plain, batch, k, v, q=q, inv_freq=freq))
    turned = q4.q4_kv_append(cache, batch, k, v, q=q, inv_freq=freq, q_out=q)
    assert turned is q and torch.equal(packed[:, hq * dim:], kv)
    assert torch.equal(q4.q4_attention_paged(cache, batch, q), want)
    assert torch.equal(both[:, 0], plain.k) and torch.equal(both[:, 1], plain.v)


def test_no_new_tokens_at_all():
    """Sequences without new tokens: nothing is written, whatever rows the tensors have."""
    q4 = lib()
    batch = kv_ref.Batch([(0, 40), (0, 0), (0, 3000)], 16, pad_rows=3)
    q, k, v = make(batch, 4, 2, 128, torch.float16)
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    kc, vc = on_gpu(k), on_gpu(v)
    cache, dev = q4.KVCache(kc, vc), batch.device(q4)
    before = kc.view(torch.int16).clone()
    q4.q4_attention_paged(cache, dev, q.cuda(), out=out)
    new = torch.ones(3, 2, 128, dtype=torch.float16, device="cuda")
    q4.q4_kv_append(cache, dev, new, new, q=q.cuda(), q_out=out)
    torch.cuda.synchronize()
    assert bool((out == 5.0).all()) and torch.equal(kc.view(torch.int16), before)


def test_pages_without_a_place_are_not_seen():
    """Pages given back (-1) or outside the cache, in the middle and at the ends; a sequence that holds none."""
    q4 = lib()
    batch = kv_ref.Batch([(1, 200), (30, 200), (1, 90), (2, 60)], 16, seed=4)
    batch.table[0, 0] = -1
    batch.table[0, 5] = batch.pages
    batch.table[1, 12] = -7
    batch.table[1, 3] = 2 ** 31 - 1
    batch.table[3, :] = -1
    batch.table = batch.table[:, :13].copy()
    q, k, v = make(batch, 4, 2, 64, torch.float16)
    out = check(q4, batch, q, k, v)
    assert bool((out[int(batch.start[3]):] == 0).all())


def test_scores_far_apart():
    """Scores of thousands: the maximum is raised late and often, and one key takes all the weight."""
    q4 = lib()
    for dtype in (torch.float16, torch.bfloat16):
        batch = kv_ref.Batch([(1, 777), (20, 300)], 16, seed=6)
        q, k, v = make(batch, 8, 2, 128, dtype, spread=60.0)
        check(q4, batch, q, k, v)
        # rising scores: every step raises the maximum
        q, k, v = make(batch, 8, 2, 128, dtype)
        ramp = torch.zeros(batch.pages, batch.page)
        for b in range(2):
            for p, page, slot in batch.places(b):
                ramp[page, slot] = p / 4.0
        k[..., 0] = torch.where(torch.isfinite(k[..., 0]), ramp[:, None, :].to(dtype), k[..., 0])
        q[..., 0] = 12.0
        check(q4, batch, q, k, v)


def test_nan_and_infinity_stay_in_their_rows():
    q4 = lib()
    batch = kv_ref.Batch([(20, 120)], 16, seed=7)
    q, k, v = make(batch, 4, 2, 64, torch.float16)
    clean = check(q4, batch, q, k, v).clone()
    q2 = q.clone()
    q2[3, 1] = math.nan
    out = check_rows(q4, batch, q2, k, v)
    assert bool(torch.isnan(out[3, 1]).all())
    out[3, 1] = clean[3, 1]
    assert torch.equal(out, clean)


def test_nan_in_keys_a_row_does_not_see():
    """A new token whose key and value are NaN or infinite: the rows before it do not change."""
    q4 = lib()
    for n, c in ((20, 120), (130, 300)):
        batch = kv_ref.Batch([(n, c)], 16, seed=7)
        for bad in (math.nan, math.inf):
            q, k, v = make(batch, 4, 2, 64, torch.float16)
            clean = check(q4, batch, q, k, v).clone()
            p = c - n + 9
            page, slot = int(batch.table[0, p // 16]), p % 16
            k[page, :, slot, 5] = bad
            v[page, :, slot, 7] = bad
            out = check_rows(q4, batch, q, k, v)
            assert torch.equal(out[:9], clean[:9])
            assert not bool(torch.isfinite(out[9:, :, 7]).any()) or bad == math.inf
            # windows: the rows behind it do not see it either
            clean = check_rows(q4, batch, q, torch.where(torch.isfinite(k), k, torch.zeros_like(k)),
                               torch.where(torch.isfinite(v), v, torch.zeros_like(v)), window=4)
            out = check_rows(q4, batch, q, k, v, window=4)
            assert torch.equal(out[:9], clean[:9]) and torch.equal(out[13:], clean[13:])


def check_rows(q4, batch, q, k, v, window=0):
    out = q4.q4_attention_paged(q4.KVCache(on_gpu(k), on_gpu(v)), batch.device(q4), q.cuda(), window=window)
    torch.cuda.synchronize()
    return out


def test_strided_queries_and_outputs():
    q4 = lib()
    batch = kv_ref.Batch([(3, 50), (1, 20)], 16, seed=8)
    q, k, v = make(batch, 8, 2, 64, torch.bfloat16)
    want = check(q4, batch, q, k, v)
    cache, dev = q4.KVCache(on_gpu(k), on_gpu(v)), batch.device(q4)
    packed = torch.zeros(4, 12 * 64, dtype=torch.bfloat16, device="cuda")
    packed[:, 128:640] = q.cuda().reshape(4, 512)
    out = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    assert torch.equal(q4.q4_attention_paged(cache, dev, packed[:, 128:640].view(4, 8, 64), out=out), want)


def test_workspace_and_stream():
    """A workspace of the caller's with other data in it, and a call on a stream that is not the current one."""
    q4 = lib()
    batch = kv_ref.Batch([(1, 3000), (5, 2000)], 16, seed=9)
    q, k, v = make(batch, 8, 2, 128, torch.float16)
    want = check(q4, batch, q, k, v)
    cache, dev, dq = q4.KVCache(on_gpu(k), on_gpu(v)), batch.device(q4), q.cuda()
    need = q4.attention_workspace_bytes(cache, dev, 8, batch.tokens)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaNs
    assert torch.equal(q4.q4_attention_paged(cache, dev, dq, workspace=ws), want)
    if need:
        with pytest.raises(q4.Q4Error):
            q4.q4_attention_paged(cache, dev, dq, workspace=ws[: need - 16])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = q4.q4_attention_paged(cache, dev, dq, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_captured_with_new_lengths():
    """A graph of a decode step (append and attention) replayed with other lengths, tables and tokens in the same
    tensors, a second graph of the same cache in between and eager work too: every replay as the eager call."""
    q4 = lib()
    page, hk, hq, dim = 16, 2, 8, 128
    steps = [[(1, 40), (1, 700), (1, 3)], [(1, 41), (1, 701), (1, 4)], [(1, 1), (1, 2000), (0, 77)], [(1, 500), (0, 0), (1, 16)]]
    batches = [kv_ref.Batch(lens, page, spare=300, seed=i, columns=130) for i, lens in enumerate(steps)]
    pages = max(b.pages for b in batches)
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(pages, hk, page, dim, generator=g).half().cuda() for _ in range(2))
    cache = q4.KVCache(kc, vc)
    table, start, ctx = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((3, 130), (4,), (3,)))
    batch = q4.KVBatch(table, start, ctx, max_query_len=1, max_context_len=2080)
    packed = torch.zeros(3, (hq + 2 * hk) * dim, device="cuda")
    q, k, v = packed.view(3, -1, dim).split([hq, hk, hk], 1)
    freq, _ = q4.rope_frequencies(dim)
    out, out2 = (torch.zeros(3, hq, dim, dtype=torch.float16, device="cuda") for _ in range(2))

    def step(to):
        turned = q4.q4_kv_append(cache, batch, k, v, q=q, inv_freq=freq)
        q4.q4_attention_paged(cache, batch, turned, out=to)

    def load(i):
        b = batches[i % len(steps)]
        table.copy_(torch.from_numpy(b.table))
        start.copy_(torch.from_numpy(b.start))
        ctx.copy_(torch.tensor(b.ctx, dtype=torch.int32))
        packed.copy_(torch.randn(packed.shape, generator=g))

    load(0)
    step(out)
    torch.cuda.synchronize()
    graphs = []
    for to in (out, out2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(to)
        graphs.append(graph)
    for i in range(8):
        load(i)
        out.fill_(3.0)
        out2.fill_(3.0)
        kc0, vc0 = kc.clone(), vc.clone()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        got_k, got_v = kc.clone(), vc.clone()
        kc.copy_(kc0)
        vc.copy_(vc0)
        want = torch.full_like(out, 3.0)
        step(want)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want), i
        assert torch.equal(kc, got_k) and torch.equal(vc, got_v), i


def test_layer_step_with_the_products():
    """A decoder layer's attention block as a program runs it: the q, k and v products (GEMV of one token, small-M of
    a chunk) into packed rows, append with rotation, attention, the o product; against the same chain in 64 bits from
    the products' own outputs on."""
    import oracle
    import synth
    q4 = lib()
    hidden, hq, hk, dim, page = 512, 8, 2, 64, 16
    rows = (hq + 2 * hk) * dim
    wq = synth.q4_0(synth.DEFAULT_SEED, 7001, rows, hidden)
    wo = synth.q4_0(synth.DEFAULT_SEED, 7002, hidden, hq * dim)
    dwq, dwo = torch.from_numpy(wq).cuda(), torch.from_numpy(wo).cuda()
    kc, vc = (torch.zeros(12, hk, page, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = q4.KVCache(kc, vc)
    freq, _ = q4.rope_frequencies(dim)
    table = torch.tensor([[7, 2, 9, 4, 0, 11]], dtype=torch.int32, device="cuda")
    done = 0
    keys, values = [], []
    for n in (16, 1, 1, 5, 1):  # a chunk of the prompt, decode, a draft's verify
        x = torch.from_numpy(synth.f16_normal(synth.DEFAULT_SEED, 7100 + done, n * hidden).reshape(n, hidden)).cuda()
        packed = q4.q4_0_gemv(dwq, x[0].contiguous()).view(1, -1) if n == 1 else q4.q4_0_gemm_smallm(dwq, x)
        q, k, v = packed.view(n, -1, dim).split([hq, hk, hk], 1)
        batch = q4.KVBatch(table, torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                           torch.tensor([done + n], dtype=torch.int32, device="cuda"), max_query_len=n, max_context_len=96)
        turned = q4.q4_kv_append(cache, batch, k, v, q=q, inv_freq=freq)
        out = q4.q4_attention_paged(cache, batch, turned)
        y = q4.q4_0_gemv(dwo, out.view(-1)) if n == 1 else q4.q4_0_gemm_smallm(dwo, out.view(n, -1))
        torch.cuda.synchronize()
        # the oracle's cache: the same roundings to 16 bits as the operators document
        pos = torch.arange(done, done + n)
        keys.append(kv_ref.rotate(k.double().cpu(), pos, freq.cpu(), "half").half())
        values.append(v.half().cpu())
        at = [(int(table[0, p // page]), p % page) for p in range(done + n)]
        got_k = torch.stack([kc[a, :, s] for a, s in at]).cpu()
        got_v = torch.stack([vc[a, :, s] for a, s in at]).cpu()
        assert torch.equal(got_v, torch.cat(values))
        want_k = torch.cat(keys).double()
        # a value next to a border between two halves may go to the other one: a step of it
        assert bool(((got_k.double() - want_k).abs() <= 2.0 ** -10 * want_k.abs() + 2.0 ** -24).all())
        ref = kv_ref.Batch([(n, done + n)], page)
        ref.table, ref.pages = table.cpu().numpy(), 12
        want, _, bound, _ = kv_ref.attention(turned.cpu(), kc.cpu(), vc.cpu(), ref, dim ** -0.5, 0)
        assert bool(((out.double().cpu() - want).abs() <= bound).all())
        y_ref, a_ref = oracle.gemm_rows(wo, hq * dim, out.cpu().numpy().reshape(n, -1))
        assert bool((np.abs(y.cpu().numpy().reshape(n, -1) - y_ref.reshape(n, -1)) <= oracle.TOL * a_ref.reshape(n, -1)).all())
        done += n


def test_far_offsets():
    """A cache of more than 4 GiB: pages at its end and its beginning."""
    q4 = lib()
    page, hk, dim = 128, 8, 128
    pages = (1 << 32) // (page * hk * dim * 2) + 40
    k = torch.zeros(pages, hk, page, dim, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    batch = kv_ref.Batch([(1, 500), (33, 700)], page, spare=0, seed=10)
    q, ks, vs = make(batch, hk, hk, dim, torch.float16)
    want, _, bound, _ = kv_ref.attention(q, ks, vs, batch, dim ** -0.5, 0)
    to = np.where(np.arange(batch.pages) % 2 == 0, pages - 1 - np.arange(batch.pages), np.arange(batch.pages))
    k[torch.from_numpy(to).cuda()] = ks.cuda()
    v[torch.from_numpy(to).cuda()] = vs.cuda()
    batch.table = np.where(batch.table >= 0, to[batch.table], -1).astype(np.int32)
    out = q4.q4_attention_paged(q4.KVCache(k, v), batch.device(q4), q.cuda()).double().cpu()
    assert bool(((out - want).abs() <= bound).all())


def test_same_results_twice():
    q4 = lib()
    batch = kv_ref.Batch([(1, 4000), (1, 100), (50, 600)], 64, seed=11)
    q, k, v = make(batch, 32, 8, 128, torch.bfloat16)
    cache, dev, dq = q4.KVCache(on_gpu(k), on_gpu(v)), batch.device(q4), q.cuda()
    first = q4.q4_attention_paged(cache, dev, dq)
    for _ in range(5):
        assert torch.equal(q4.q4_attention_paged(cache, dev, dq), first)

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

"""The cache operators at the ends of their ranges: batches of very many sequences, very many tokens or items."""
import numpy as np
import pytest
import torch

from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def many(seqs, seed, most=2):
    """0 .. most new tokens a sequence and contexts of one page, a page each: starts, contexts, rows' sequences and
    positions, and the table."""
    rng = np.random.default_rng(seed)
    new = rng.integers(0, most + 1, seqs)
    new[rng.integers(0, seqs, 3)] = 0
    new[-1] = 1
    ctx = np.minimum(new + rng.integers(0, 8 - most, seqs), 8)
    start = np.concatenate([[0], np.cumsum(new)])
    seq = np.repeat(np.arange(seqs), new)
    pos = ctx[seq] - new[seq] + np.arange(start[-1]) - start[seq]
    table = rng.permutation(seqs).astype(np.int32)[:, None]
    return start.astype(np.int32), ctx.astype(np.int32), seq, pos, table


def on(q4, start, ctx, table, **hints):
    return q4.KVBatch(*(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (table, start, ctx)), **hints)


@pytest.mark.parametrize("seqs", [64, 65, 4096, 4097, 300000])
def test_append_finds_its_sequence_among_many(seqs):
    """Every token finds its sequence in a few loads (a walk through all of them, by every token, would not end in a
    time one could wait for at the sizes that are allowed)."""
    q4 = lib()
    say("append, sequences", seqs)
    start, ctx, seq, pos, table = many(seqs, seqs)
    t = int(start[-1])
    k = torch.arange(t * 8, dtype=torch.int32).view(t, 1, 8).remainder(2039).half().cuda()
    kc, vc = (torch.full((seqs, 1, 8, 8), -1.0, dtype=torch.float16, device="cuda") for _ in range(2))
    want = kc.clone()
    want[torch.from_numpy(table[seq, 0]).long().cuda(), 0, torch.from_numpy(pos).cuda()] = k[:, 0]
    q4.q4_kv_append(q4.KVCache(kc, vc), on(q4, start, ctx, table), k, -k)
    torch.cuda.synchronize()
    assert torch.equal(kc, want)
    assert torch.equal(vc, torch.where(want == -1.0, want, -want))


def uniform(q4, new, ctx, hq, hk, dim, slots=65536, **hints):
    """Attention with queries of 0, all sequences in one page: a row's output is the mean of the values
    it sees, every weight alike and so exact.  Checks it, and returns the workspace that the call needs.

    An output is off by its rounding, half a step, and by the 32-bit sum of at most 400 values below 8 in each of
    which a rounding of 2^-24 of a partial sum is made: 400 * 2^-24 * 8 < 2^-12."""
    rng = np.random.default_rng(len(new))
    k, v = (torch.from_numpy(rng.normal(0, 1, (1, hk, slots, dim)).clip(-7, 7)).half().cuda() for _ in range(2))
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    seq = np.repeat(np.arange(len(new)), new)
    sees = ctx[seq] - new[seq] + np.arange(start[-1]) - start[seq] + 1
    assert sees.max() <= 400
    batch = on(q4, start, ctx.astype(np.int32), np.zeros((len(new), 1), dtype=np.int32), **hints)
    t = int(start[-1])
    out = torch.full((t + 3, hq, dim), 5.0, dtype=torch.float16, device="cuda")
    cache = q4.KVCache(k, v)
    q4.q4_attention_paged(cache, batch, torch.zeros_like(out), out=out)
    torch.cuda.synchronize()
    n = torch.from_numpy(sees).cuda()
    mean = v[0, :, :400].double().cumsum(1) / torch.arange(1, 401, device="cuda")[:, None]
    mean = torch.cat((torch.zeros_like(mean[:, :1]), mean), 1)  # none: 0
    want = mean[:, n.clamp(min=0)].transpose(0, 1).repeat_interleave(hq // hk, 1)
    assert bool(((out[:t].double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -12).all())
    assert bool((out[t:] == 5.0).all())
    return q4.attention_workspace_bytes(cache, batch, hq, t + 3)


@pytest.mark.parametrize("seqs,most,hint,whole", [
    (65, 2, 1000, True), (4097, 2, 1000, True), (20000, 1, 1000, True), (130, 40, 1000, True), (4200, 17, 1000, True),
    (65, 2, 65536, False), (4097, 2, 100, False), (130, 40, 65536, False)])
def test_items_of_many_sequences(seqs, most, hint, whole):
    """Items find their sequence among many, most of the sequences' rows not a multiple of an item's."""
    q4 = lib()
    say("attention, sequences", seqs, most)
    rng = np.random.default_rng(seqs)
    new = rng.integers(0, most + 1, seqs)
    new[[0, seqs // 2]] = 0
    ctx = np.maximum(new + rng.integers(-2, 300, seqs), 0)
    # the hint decides whether items are taken whole
    assert (uniform(q4, new, ctx, 6, 2, 64, max_query_len=most, max_context_len=hint) == 0) == whole


def test_more_items_than_a_launch_has_workgroups():
    """2^23 workgroups of 512 threads are one too many for a launch; with one item each this call has 200 more."""
    q4 = lib()
    seqs, hk = 131073, 64
    new = np.ones(seqs, dtype=np.int64)
    ctx = np.random.default_rng(5).integers(0, 60, seqs)
    assert uniform(q4, new, ctx, hk, hk, 64, slots=1024, max_query_len=1, max_context_len=1024) == 0


def test_more_tokens_than_a_launch_has_workgroups():
    """2^24 workgroups of 256 threads, of 4 tokens each, are one too many for a launch."""
    q4 = lib()
    t, period = (1 << 26) + 5, 1 << 20
    g = torch.Generator().manual_seed(1)
    x = torch.randn(period, 1, 2, generator=g).half().cuda()
    pos = torch.randint(0, 1 << 20, (period,), generator=g, dtype=torch.int32).cuda()
    freq = torch.tensor([0.25], dtype=torch.float64, device="cuda")
    want = q4.q4_rope(x, pos, freq)
    got = q4.q4_rope(x.repeat(65, 1, 1)[:t], pos.repeat(65)[:t], freq)
    torch.cuda.synchronize()
    assert torch.equal(got[: 64 * period].view(64, period, 2), want.view(1, period, 2).expand(64, -1, -1))
    assert torch.equal(got[64 * period :], want[:5])


@pytest.mark.parametrize("seqs", [0, 3])
def test_a_step_without_tokens(seqs):
    """Token tensors without rows, of a batch with or without sequences: outputs without rows, the cache as it was."""
    q4 = lib()
    kc, vc = (torch.full((2, 2, 8, 64), 3.0, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = q4.KVCache(kc, vc)
    batch = on(q4, np.zeros(seqs + 1, dtype=np.int32), np.full(seqs, 5, dtype=np.int32), np.zeros((seqs, 1), dtype=np.int32))
    freq, _ = q4.rope_frequencies(64)
    kv = torch.empty((0, 2, 64), device="cuda")
    q = torch.empty((0, 4, 64), device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert q4.q4_rope(q, none, freq).shape == (0, 4, 64)
    assert q4.q4_kv_append(cache, batch, kv, kv, inv_freq=freq) is None
    turned = q4.q4_kv_append(cache, batch, kv, kv, q=q, inv_freq=freq, positions=none)
    assert turned.shape == (0, 4, 64) and turned.dtype == torch.float16
    out = torch.empty_like(turned)
    assert q4.attention_workspace_bytes(cache, batch, 4, 0) == 0
    assert q4.q4_attention_paged(cache, batch, turned).shape == (0, 4, 64)
    assert q4.q4_attention_paged(cache, batch, turned, out=out, lse=torch.empty((0, 4), device="cuda")) is out
    torch.cuda.synchronize()
    assert bool((kc == 3.0).all()) and bool((vc == 3.0).all())
    with pytest.raises(ValueError):
        q4.q4_rope(q, none, freq, layout="other")  # what is wrong stays wrong
    with pytest.raises(ValueError):
        q4.q4_kv_append(cache, batch, kv, kv, positions=torch.empty(1, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("hint", [2 ** 31, 2 ** 32 + 5, 2 ** 40])
def test_hints_past_32_bits(hint):
    """A longest context or query beyond what 32 bits hold is a hint as any other (its low bits would be negative, or
    a few tokens)."""
    q4 = lib()
    start, ctx = np.array([0, 2, 3], dtype=np.int32), np.array([5, 7], dtype=np.int32)
    table = np.array([[0], [1]], dtype=np.int32)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(2, 1, 8, 64, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(3, 2, 64, generator=g).half().cuda()
    cache = q4.KVCache(k, v)
    want = q4.q4_attention_paged(cache, on(q4, start, ctx, table), q)
    batch = on(q4, start, ctx, table, max_query_len=hint, max_context_len=hint)
    assert batch.desc.max_query == batch.desc.max_context == 2 ** 31 - 1
    assert torch.equal(q4.q4_attention_paged(cache, batch, q), want)

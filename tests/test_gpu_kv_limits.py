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

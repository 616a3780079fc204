"""Attention where one key outweighs a great many others, each with a weight of 2^-25 of its own."""
import math

import pytest
import torch

from gpu_util import lib, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("rows,pad", [(1, 0), (24, 0), (64, 0), (200, 70000)])  # items of 16, 32, 64 and 128 rows
def test_a_heavy_key_and_a_long_tail(rows, pad, dim, dtype):
    """Key 0 has the score 25.125 (as a power of 2) and the value 0, the others 0 and 1: with N of them a row is
    N w / (1 + N w), w = 2^-25.125.

    How far it may be off: in binary16 a weight is off by half of 2^-24 at most, and the largest weight is held as 2^7
    at least, so by 2^-32 of that one, in the products and in the sum: 2 N 2^-32.  In bfloat16 by 2^-8 of itself.  The
    sum of weights in 32 bits goes pair by pair, in two lanes for a row of 128 (in more for fewer rows): N / 4 roundings
    of at most half of 2^-23 (the sum is 1 and a little), N 2^-26.  The exponent is off by less than 2^-18 (25 in 32 bits, the scale), the
    output by its own rounding.  With the largest weight as 1, binary16 loses the whole tail of a wave's keys."""
    q4 = lib()
    say("tail", rows, dim, dtype)
    ctx = 131072
    k, v = (torch.zeros(2, 1, 65536, dim, dtype=dtype, device="cuda") for _ in range(2))
    k[1, 0, 0, dim // 2] = 25.125
    v[:] = 1.0
    v[1, 0, 0] = 0.0
    q = torch.zeros(rows + pad, 1, dim, dtype=dtype, device="cuda")
    q[:, :, dim // 2] = 1.0
    batch = q4.KVBatch(torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                       torch.tensor([ctx], dtype=torch.int32, device="cuda"),
                       max_query_len=rows, max_context_len=rows)  # the hint: items are taken whole, in one sum
    cache = q4.KVCache(k, v)
    assert q4.attention_workspace_bytes(cache, batch, 1, rows + pad) == 0
    lse = torch.empty(rows + pad, 1, device="cuda")
    out = q4.q4_attention_paged(cache, batch, q, scale=math.log(2.0), lse=lse)[:rows].double().cpu()
    n = torch.arange(ctx - rows, ctx, dtype=torch.float64)
    tail = n * 2.0 ** -25.125
    step = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    weights = n * (2.0 ** -31 if dtype == torch.float16 else 0) + tail * (0 if dtype == torch.float16 else 2 * step)
    total = n * 2.0 ** -26
    want = tail / (1 + tail)
    assert bool(((out - want[:, None, None]).abs() <= ((step + 2.0 ** -17 + total) * want + weights)[:, None, None]).all())
    want = 25.125 * math.log(2.0) + torch.log1p(tail)
    off = (lse[:rows].double().cpu()[:, 0] - want).abs()
    assert bool((off <= weights + total + 2.0 ** -17 * tail + 2.0 ** -22 * want).all())

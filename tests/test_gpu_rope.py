"""Rotary positions and the append of new keys and values to a paged cache, against the same in 64 bits."""
import numpy as np
import pytest
import torch

import kv_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu


def close(got, want, bound, what=""):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d outside, worst %g of the bound" % (what, int(bad.sum()), float((err / bound).max()))


@pytest.mark.parametrize("tokens,heads,dim,rot,layout,src,dst", [
    (1, 40, 128, 128, "half", torch.float16, torch.float16),
    (3, 1, 2, 2, "half", torch.float32, torch.float32),
    (5, 3, 80, 32, "half", torch.bfloat16, torch.bfloat16),
    (9, 7, 96, 96, "interleaved", torch.float16, torch.float32),
    (130, 5, 256, 64, "interleaved", torch.float32, torch.bfloat16),
    (33, 2, 67, 22, "half", torch.float16, torch.float16),       # odd head, no vector path
    (33, 2, 67, 22, "interleaved", torch.bfloat16, torch.float16),
    (4, 2, 1024, 1024, "half", torch.float32, torch.float16),
    (1027, 32, 128, 128, "half", torch.bfloat16, torch.bfloat16),
])
def test_rope(tokens, heads, dim, rot, layout, src, dst):
    q4 = lib()
    say("rope", tokens, heads, dim, rot, layout, src, dst)
    g = torch.Generator().manual_seed(tokens * dim + rot)
    x = torch.randn(tokens, heads, dim, generator=g).to(src)
    pos = torch.randint(-50, 1 << 20, (tokens,), generator=g, dtype=torch.int32)
    freq, _ = q4.rope_frequencies(rot, 1e6, device="cpu")
    got = q4.q4_rope(x.cuda(), pos.cuda(), freq.cuda(), layout, mscale=1.25, out=torch.empty(x.shape, dtype=dst, device="cuda"))
    close(got, kv_ref.rotate(x.double(), pos, freq, layout, 1.25), kv_ref.rotate_bound(x.double(), pos, freq, layout, dst, 1.25))


def test_rope_strided_and_in_place():
    q4 = lib()
    g = torch.Generator().manual_seed(5)
    packed = torch.randn(37, 10 * 64, generator=g).half()
    pos = torch.arange(37, dtype=torch.int32)
    freq, _ = q4.rope_frequencies(64, device="cpu")
    want = kv_ref.rotate(packed[:, :256].reshape(37, 4, 64).double(), pos, freq, "half")
    dev = packed.cuda()
    part = dev[:, :256].view(37, 4, 64)
    out = q4.q4_rope(part, pos.cuda(), freq.cuda())
    back = q4.q4_rope(part, pos.cuda(), freq.cuda(), out=part)
    assert back is part
    assert torch.equal(part, out)
    assert torch.equal(dev[:, 256:].cpu(), packed[:, 256:])  # the rest of the packed rows is untouched
    close(out, want, kv_ref.rotate_bound(packed[:, :256].reshape(37, 4, 64).double(), pos, freq, "half", torch.float16))
    # heads outside, tokens inside, off 16-byte alignment
    odd = torch.zeros(4 * 37 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(4, 37, 64).transpose(0, 1)
    assert torch.equal(q4.q4_rope(packed.cuda()[:, :256].view(37, 4, 64), pos.cuda(), freq.cuda(), out=odd), out)


def test_rope_gradient():
    """The gradient of sum(w * rope(x)) is w turned back; against differences of the 64-bit form."""
    q4 = lib()
    g = torch.Generator().manual_seed(6)
    x, w = torch.randn(3, 2, 16, generator=g).double(), torch.randn(3, 2, 16, generator=g)
    pos = torch.tensor([0, 7, 100], dtype=torch.int32)
    freq, _ = q4.rope_frequencies(8, device="cpu")
    for layout in ("half", "interleaved"):
        grad = q4.q4_rope(w.cuda(), (-pos).cuda(), freq.cuda(), layout).cpu().double()
        for at in ((0, 0, 0), (1, 1, 5), (2, 0, 3), (2, 1, 12)):
            up, down = x.clone(), x.clone()
            up[at] += 0.5
            down[at] -= 0.5  # the form is linear: a difference is exact up to rounding
            diff = ((kv_ref.rotate(up, pos, freq, layout) - kv_ref.rotate(down, pos, freq, layout)) * w.double()).sum()
            assert abs(float(grad[at] - diff)) <= 2.0 ** -19 * float(w[at[:2]].abs().sum())


def test_far_positions_keep_their_angle():
    """One pair, position 2^24 - 1 and frequency 1: the angle in 32 bits would be off by up to a unit."""
    q4 = lib()
    x = torch.tensor([[[1.0, 0.0]]], device="cuda")
    for p in (16777215, -16777215, 1 << 30):
        got = q4.q4_rope(x, torch.tensor([p], dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.float64, device="cuda"))
        want = [np.cos(float(p)), np.sin(float(p))]
        assert np.allclose(got.cpu().numpy()[0, 0], want, atol=2.0 ** -20, rtol=0)


@pytest.mark.parametrize("lens,page,hq,hk,dim,rot,layout,src,dst", [
    ([(1, 170)], 16, 32, 8, 128, 128, "half", torch.float32, torch.float16),
    ([(1, 1), (1, 64), (1, 65), (1, 500)], 64, 8, 8, 64, 64, "half", torch.float16, torch.float16),
    ([(5, 5), (0, 30), (17, 40), (0, 0), (1, 9)], 8, 6, 2, 96, 48, "interleaved", torch.bfloat16, torch.bfloat16),
    ([(3, 12), (40, 100)], 24, 3, 3, 20, 6, "half", torch.float32, torch.bfloat16),  # no vector path
    ([(1, c) for c in range(1, 130)], 16, 4, 1, 64, 0, "half", torch.float16, torch.float16),  # no rotation
])
@pytest.mark.parametrize("slots_first", [False, True])
def test_append(lens, page, hq, hk, dim, rot, layout, src, dst, slots_first):
    q4 = lib()
    say("append", lens[:5], page, hq, hk, dim, rot, layout, src, dst, slots_first)
    batch = kv_ref.Batch(lens, page, seed=3, pad_rows=3)
    g = torch.Generator().manual_seed(page + dim)
    packed = torch.randn(batch.tokens, (hq + 2 * hk) * dim, generator=g).to(src)
    q, k, v = packed.view(batch.tokens, -1, dim).split([hq, hk, hk], 1)
    shape = (batch.pages, page, hk, dim) if slots_first else (batch.pages, hk, page, dim)
    order = (0, 2, 1, 3) if slots_first else (0, 1, 2, 3)
    kc, vc = (torch.randn(shape, generator=g).to(dst).cuda().permute(order) for _ in range(2))
    want_k, want_v = kc.double().cpu(), vc.double().cpu()
    bound_k = torch.zeros_like(want_k)
    freq = q4.rope_frequencies(rot, 1e4, device="cpu")[0] if rot else torch.zeros(0, dtype=torch.float64)
    dev = packed.cuda().view(batch.tokens, -1, dim)
    dq, dk, dv = dev.split([hq, hk, hk], 1)
    out = torch.full((batch.tokens, hq, dim), 7.0, dtype=dst, device="cuda")
    got = q4.q4_kv_append(q4.KVCache(kc, vc), batch.device(q4), dk, dv, q=dq, inv_freq=freq.cuda() if rot else None,
                          layout=layout, mscale=1.0, q_out=out)
    torch.cuda.synchronize()
    for b in range(len(lens)):
        n, c = lens[b]
        rows = slice(int(batch.start[b]), int(batch.start[b + 1]))
        pos = torch.arange(c - n, c)
        close(got[rows], kv_ref.rotate(q[rows].double(), pos, freq, layout),
              kv_ref.rotate_bound(q[rows].double(), pos, freq, layout, dst), "q of %d" % b)
        kr = kv_ref.rotate(k[rows].double(), pos, freq, layout)
        kb = kv_ref.rotate_bound(k[rows].double(), pos, freq, layout, dst)
        for i in range(n):
            at, slot = int(batch.table[b, (c - n + i) // page]), (c - n + i) % page
            want_k[at, :, slot], bound_k[at, :, slot] = kr[i], kb[i]
            want_v[at, :, slot] = v[rows][i].to(dst).double()
    err = (kc.double().cpu() - want_k).abs()
    assert bool((err <= bound_k).all())  # bound 0 where nothing was appended
    assert torch.equal(vc.double().cpu(), want_v)
    assert bool((out[batch.tokens - 3:] == 7.0).all())  # rows behind the last sequence


def test_append_without_a_place():
    """Positions below 0, beyond the table or in a page outside the cache are not written; their queries still turn."""
    q4 = lib()
    page, hk, dim = 8, 2, 64
    batch = kv_ref.Batch([(6, 3), (4, 20), (4, 12), (2, 16)], page, seed=1)
    batch.table[2, 1] = -1
    batch.table[3, 1] = batch.pages
    table = batch.table[:, :2].copy()  # sequence 1's tokens 16 .. 19 lie beyond two pages
    batch.table = table
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn(batch.tokens, h, dim, generator=g).half().cuda() for h in (hk, hk, 4))
    kc = torch.full((batch.pages, hk, page, dim), 9.0, dtype=torch.float16, device="cuda")
    vc = kc.clone()
    freq, _ = q4.rope_frequencies(dim)
    out = q4.q4_kv_append(q4.KVCache(kc, vc), batch.device(q4), k, v, q=q, inv_freq=freq)
    pos = torch.tensor([p for (n, c) in ((6, 3), (4, 20), (4, 12), (2, 16)) for p in range(c - n, c)], dtype=torch.int32)
    assert torch.equal(out, q4.q4_rope(q, pos.cuda(), freq))
    turned = q4.q4_rope(k, pos.cuda(), freq)
    want = torch.full_like(kc, 9.0)
    for i in range(3):  # only sequence 0's positions 0, 1, 2 have a place
        want[int(table[0, 0]), :, i] = turned[3 + i]
    assert torch.equal(kc, want)
    assert int((vc != 9.0).any(-1).sum()) == 3 * hk


def test_append_with_given_positions():
    q4 = lib()
    page, hk, dim = 16, 2, 64
    batch = kv_ref.Batch([(5, 20)], page)
    g = torch.Generator().manual_seed(2)
    k = torch.randn(5, hk, dim, generator=g).bfloat16().cuda()
    pos = torch.tensor([5, 100000, 3, 0, -4], dtype=torch.int32, device="cuda")
    freq, _ = q4.rope_frequencies(dim)
    kc, vc = (torch.zeros(batch.pages, hk, page, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert q4.q4_kv_append(q4.KVCache(kc, vc), batch.device(q4), k, k, inv_freq=freq, positions=pos) is None
    turned = q4.q4_rope(k, pos, freq)
    for i in range(5):
        assert torch.equal(kc[int(batch.table[0, (15 + i) // page]), :, (15 + i) % page], turned[i])

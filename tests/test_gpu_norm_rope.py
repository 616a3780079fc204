"""q4_norm_rope and q4_kv_append_norm against the norm and the rotation in 64 bits."""
import pytest
import torch

import kv_ref
import step_ref
from gpu_util import lib, say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def check(got, x, gain, eps, pos, freq, layout, mscale=1.0):
    f = None if freq is None else freq.cpu()
    x, pos, g = x.double().cpu(), None if pos is None else pos.cpu(), None if gain is None else gain.cpu()
    want = step_ref.norm(x, g, eps)
    if freq is not None:
        want = kv_ref.rotate(want, pos, f, layout, mscale)
    bound = step_ref.norm_rope_bound(x, g, eps, pos, f, layout, got.dtype, mscale)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("src,dst", [(F16, F16), (BF16, BF16), (F32, F16), (F32, BF16), (F32, F32), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("t,h,d,rot", [(1, 1, 64, 64), (1, 40, 128, 128), (5, 3, 128, 64), (9, 8, 256, 256), (3, 5, 96, 48), (2, 2, 1024, 1024),
                                       (4, 3, 1024, 512), (3, 2, 1024, 0), (2, 3, 8, 0), (7, 2, 80, 80), (6, 3, 90, 34), (3, 4, 7, 6), (2, 2, 1, 0),
                                       (2, 3, 513, 512), (3, 3, 1023, 2), (130, 7, 128, 128)])
def test_shapes(t, h, d, rot, layout, src, dst):
    """Heads of every path: one unit a lane and several, whole and partly turned or not at all, of 16 bytes and single
    elements, odd sizes."""
    q4 = lib()
    g = torch.Generator(device="cuda").manual_seed(d + rot)
    packed = torch.randn(t, (h + 2) * d, device="cuda", generator=g).mul_(3.0).to(src)
    x = packed[:, d : (h + 1) * d].view(t, h, d)
    gain = (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(dst)
    pos = torch.randint(0, 1 << 20, (t,), device="cuda", generator=g, dtype=torch.int32)
    freq = q4.rope_frequencies(rot, 1e6)[0] if rot else None
    out = torch.empty(t, h, d, dtype=dst, device="cuda")
    q4.q4_norm_rope(x, gain, eps=1e-6, positions=pos if rot else None, inv_freq=freq, layout=layout, out=out)
    check(out, x, gain, 1e-6, pos if rot else None, freq, layout)


@pytest.mark.parametrize("kind", [F16, BF16, F32])
def test_gains_eps_scale(kind):
    """Gains of every type and none, eps 0 and large, a factor on what turns, heads of zeros, small and large values."""
    q4 = lib()
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(6, 4, 128, device="cuda", generator=g)
    x[1] *= 1e-3
    x[2] *= 2e4
    x[3, 0] = 0.0
    x[3, 1, 5:] = 0.0
    pos = torch.tensor([0, 1, -3, 7, 131071, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    freq, _ = q4.rope_frequencies(64, 1e4)
    for gain in (None, torch.randn(128, device="cuda", generator=g).to(kind)):
        for eps in (1e-6, 1e-2, 3.0):
            out = torch.empty(6, 4, 128, dtype=F32, device="cuda")
            q4.q4_norm_rope(x, gain, eps, pos, freq, mscale=1.25, out=out)
            # far positions: the angle's last bits in 64 bits
            check(out[:5], x[:5], gain, eps, pos[:5], freq, "half", 1.25)
            assert bool((out[3, 0] == 0).all())
    some = x[[0, 1, 2, 4]].contiguous()
    out = q4.q4_norm_rope(some, None, 0.0)
    check(out, some, None, 0.0, None, None, "half")


def test_in_place_strides_and_broadcast():
    """out is x itself, a part of packed rows; heads that are one head; strides that are odd; all as of whole tensors."""
    q4 = lib()
    g = torch.Generator(device="cuda").manual_seed(4)
    freq, _ = q4.rope_frequencies(128)
    pos = torch.randint(0, 5000, (37,), device="cuda", generator=g, dtype=torch.int32)
    gain = torch.randn(128, device="cuda", generator=g).half()
    for width in (10 * 128, 10 * 128 + 1, 10 * 128 + 8):
        packed = torch.randn(37, width, device="cuda", generator=g).half()
        x = packed[:, 128 : 9 * 128].view(37, 8, 128)
        before = packed.clone()
        want = q4.q4_norm_rope(x.contiguous(), gain, 1e-6, pos, freq)
        q4.q4_norm_rope(x, gain, 1e-6, pos, freq, out=x)
        check(x, before[:, 128 : 9 * 128].view(37, 8, 128), gain, 1e-6, pos, freq, "half")
        if width % 8 == 0:
            assert torch.equal(x, want)
        assert torch.equal(packed[:, :128], before[:, :128]) and torch.equal(packed[:, 9 * 128:], before[:, 9 * 128:])
    one = torch.randn(37, 1, 128, device="cuda", generator=g).half().expand(37, 6, 128)
    assert torch.equal(q4.q4_norm_rope(one, gain, 1e-6, pos, freq), q4.q4_norm_rope(one.contiguous(), gain, 1e-6, pos, freq))
    assert q4.q4_norm_rope(one[:0], gain, 1e-6, pos[:0], freq).shape == (0, 6, 128)


def test_single_head_is_a_row_of_many():
    """A head's result depends on its values alone, wherever it lies and however many there are."""
    q4 = lib()
    x = torch.randn(50, 12, 128, device="cuda").half()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    freq, _ = q4.rope_frequencies(128)
    whole = q4.q4_norm_rope(x, None, 1e-6, pos, freq)
    for t, h in ((0, 0), (17, 5), (49, 11)):
        assert torch.equal(q4.q4_norm_rope(x[t : t + 1, h : h + 1].contiguous(), None, 1e-6, pos[t : t + 1], freq)[0, 0], whole[t, h])


@pytest.mark.parametrize("dim,page,src,dst,layout,rot", [(128, 16, F32, F16, "half", 128), (128, 24, BF16, BF16, "interleaved", 64), (64, 8, F16, F16, "half", 64),
                                                         (96, 32, F32, BF16, "half", 48), (256, 16, BF16, BF16, "half", 256), (80, 16, F32, F16, "interleaved", 80),
                                                         (128, 64, F16, F16, "half", 0), (33, 8, F32, F16, "half", 32)])
@pytest.mark.parametrize("lens", [[(1, 171)], [(5, 5), (0, 40), (1, 100), (30, 33), (2, 20)]])
def test_append(lens, dim, page, src, dst, layout, rot):
    """Keys normed, turned and stored, values stored, queries normed and turned; other slots and rows as they were; with
    positions of their own the angles, not the places, are theirs."""
    q4 = lib()
    say("append norm", lens, dim, page, src, dst, layout, rot)
    hq, hk = 8, 2
    batch = kv_ref.Batch(lens, page, seed=dim, pad_rows=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    n, tokens = int(batch.start[-1]), batch.tokens
    packed = torch.randn(tokens, (hq + 2 * hk) * dim, device="cuda", generator=g).to(src)
    q, k, v = packed.view(tokens, -1, dim).split([hq, hk, hk], 1)
    gains = [(1 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(dst) for _ in range(2)]
    freq = q4.rope_frequencies(rot)[0] if rot else None
    at = torch.cat([torch.arange(c - m, c) for m, c in lens] + [torch.zeros(tokens - n, dtype=torch.int64)]).to(torch.int32)
    for positions in (None, torch.randint(0, 9999, (tokens,), dtype=torch.int32, device="cuda", generator=g)):
        kc, vc = (torch.randn(batch.pages, hk, page, dim, device="cuda", generator=g).to(dst) for _ in range(2))
        before = kc.clone(), vc.clone()
        out = torch.full((tokens, hq, dim), 7.0, dtype=dst, device="cuda")
        q4.q4_kv_append_norm(q4.KVCache(kc, vc), batch.device(q4), k, v, q=q, k_gain=gains[0], q_gain=gains[1], eps=1e-5, inv_freq=freq,
                             layout=layout, positions=positions, q_out=out)
        angle = at.cuda() if positions is None else positions
        check(out[:n], q[:n], gains[1], 1e-5, angle[:n], freq, layout)
        assert bool((out[n:] == 7.0).all())
        stored, kept = torch.zeros(n, hk, dim, dtype=dst, device="cuda"), before[0].clone()
        for b in range(len(lens)):
            for p, pg, slot in batch.places(b):
                i = p - (batch.ctx[b] - batch.new[b])
                if i >= 0:
                    row = int(batch.start[b]) + i
                    stored[row] = kc[pg, :, slot]
                    kept[pg, :, slot] = kc[pg, :, slot]
                    assert torch.equal(vc[pg, :, slot], v[row].to(dst))
                    before[1][pg, :, slot] = vc[pg, :, slot]
        check(stored, k[:n], gains[0], 1e-5, angle[:n], freq, layout)
        assert torch.equal(kc, kept) and torch.equal(vc, before[1])


def test_append_without_gains_or_queries():
    q4 = lib()
    batch = kv_ref.Batch([(3, 9), (1, 1)], 8, seed=2)
    x = torch.randn(4, 4, 64, device="cuda")
    freq, _ = q4.rope_frequencies(64)
    caches = [q4.KVCache(*(torch.zeros(batch.pages, 2, 8, 64, dtype=F16, device="cuda") for _ in range(2))) for _ in range(2)]
    assert q4.q4_kv_append_norm(caches[0], batch.device(q4), x[:, :2], x[:, 2:], inv_freq=freq) is None
    ones = torch.ones(64, device="cuda")
    q = q4.q4_kv_append_norm(caches[1], batch.device(q4), x[:, :2], x[:, 2:], q=x, k_gain=ones, inv_freq=freq)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    pos = torch.tensor([6, 7, 8, 0], dtype=torch.int32, device="cuda")
    assert torch.equal(q, q4.q4_norm_rope(x, None, 1e-6, pos, freq, out=torch.empty(4, 4, 64, dtype=F16, device="cuda")))
    with pytest.raises(TypeError):
        q4.q4_kv_append_norm(caches[0], batch.device(q4), x[:, :2], x[:, 2:], q=x, k_gain=ones, q_gain=ones.half())


def test_values_that_are_not_finite():
    """NaN or an infinity in a head makes that head NaN or 0 and no other."""
    q4 = lib()
    x = torch.randn(9, 6, 128, device="cuda").half()
    want = q4.q4_norm_rope(x, None, 1e-6)
    y = x.clone()
    y[4, 2, 77] = float("nan")
    y[8, 5, 0] = float("inf")
    got = q4.q4_norm_rope(y, None, 1e-6)
    other = torch.ones(9, 6, dtype=torch.bool, device="cuda")
    other[4, 2] = other[8, 5] = False
    assert torch.equal(got[other], want[other])
    assert bool(torch.isnan(got[4, 2]).all()) and bool(torch.isnan(got[8, 5, 0]))

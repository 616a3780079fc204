"""Plain 64-bit forms of rotary positions, cache append and attention over a paged cache, one token and head after
the other, and the paged batches the tests run them on."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # of a rounding
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half the least number


def rotate(x, positions, inv_freq, layout, mscale=1.0):
    """x [T, H, D] float64 with its leading pairs turned."""
    out = x.clone()
    r = 2 * len(inv_freq)
    angle = positions.double()[:, None] * inv_freq.double()
    c, s = torch.cos(angle)[:, None, :] * mscale, torch.sin(angle)[:, None, :] * mscale
    first = slice(0, r, 2) if layout == "interleaved" else slice(0, r // 2)
    second = slice(1, r, 2) if layout == "interleaved" else slice(r // 2, r)
    out[..., first] = x[..., first] * c - x[..., second] * s
    out[..., second] = x[..., first] * s + x[..., second] * c
    return out


def rotate_bound(x, positions, inv_freq, layout, dtype, mscale=1.0):
    """How far a rotation in 32 bits, rounded once to dtype, may be from `rotate`: the sine and cosine are off by the
    angle's last bits (reduced in 64 bits: below 2^-22 in all for positions below 2^24) and by two roundings (and
    mscale's), the two products and their sum by three."""
    r = 2 * len(inv_freq)
    size = x.abs().clone()
    first = slice(0, r, 2) if layout == "interleaved" else slice(0, r // 2)
    second = slice(1, r, 2) if layout == "interleaved" else slice(r // 2, r)
    both = (x[..., first].abs() + x[..., second].abs()) * abs(mscale)
    size[..., first], size[..., second] = both, both
    exact = rotate(x, positions, inv_freq, layout, mscale)
    return HALF_STEP[dtype] * (exact.abs() + 2.0 ** -20 * size) + LEAST[dtype] + 2.0 ** -20 * size


class Batch:
    """Sequences of (new tokens, context) whose pages lie in random order in a cache with `spare` more pages."""

    def __init__(self, lens, page, spare=2, seed=0, pad_rows=0, columns=0):
        rng = np.random.default_rng(seed)
        self.new = [n for n, _ in lens]
        self.ctx = [c for _, c in lens]
        need = [-(-max(c, 0) // page) for c in self.ctx]
        self.pages = sum(need) + spare
        self.page = page
        order = rng.permutation(self.pages)
        width = max(max(need), 1, columns)
        self.table = np.full((len(lens), width), -1, dtype=np.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at : at + k]
            at += k
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.tokens = int(self.start[-1]) + pad_rows

    def device(self, q4, max_query_len=None):
        dev = "cuda"
        return q4.KVBatch(torch.from_numpy(self.table).to(dev), torch.from_numpy(self.start).to(dev),
                          torch.tensor(self.ctx, dtype=torch.int32, device=dev), max_query_len=max_query_len)

    def places(self, b):
        """(position, page, slot) of the positions of sequence b that have a place, page from its table."""
        got = []
        for p in range(max(self.ctx[b], 0)):
            if p // self.page < self.table.shape[1]:
                page = int(self.table[b, p // self.page])
                if 0 <= page < self.pages:
                    got.append((p, page, p % self.page))
        return got


def attention(q, k_cache, v_cache, batch, scale, window):
    """out, lse [T, H(, D)] in 64 bits, and how far an output in the queries' type, and an lse, may be off.

    The bound: scores are sums of D products in 32 bits (error at most (D + 4) 2^-24 of the sum of magnitudes, and
    the exponent's own rounding), so weights are off by twice that and an exponential's 2^-20 relative; every weight
    is rounded once to the type (twice half a step with the sum, plus half the least number each, the largest weight
    being at least 1 before division), the output once."""
    t, h, d = q.shape
    hk = k_cache.shape[1]
    group = h // hk
    kind = q.dtype
    step, least = HALF_STEP[kind], LEAST[kind]
    q = q.double().cpu()
    k_cache, v_cache = k_cache.double().cpu(), v_cache.double().cpu()
    out, lse = torch.zeros(t, h, d, dtype=torch.float64), torch.full((t, h), -math.inf, dtype=torch.float64)
    bound = torch.full((t, h, d), least, dtype=torch.float64)
    lse_bound = torch.zeros(t, h, dtype=torch.float64)
    for b in range(len(batch.new)):
        places = batch.places(b)
        n, c = batch.new[b], batch.ctx[b]
        if not n or not places:
            continue
        pos = torch.tensor([p for p, _, _ in places])
        pages, slots = torch.tensor([x for _, x, _ in places]), torch.tensor([s for _, _, s in places])
        row_pos = torch.arange(c - n, c)
        seen = pos[None, :] <= row_pos[:, None]
        if window:
            seen &= pos[None, :] > row_pos[:, None] - window
        rows = slice(int(batch.start[b]), int(batch.start[b + 1]))
        some = seen.any(1)
        for head in range(h):
            k = k_cache[pages, head // group, slots]
            v = v_cache[pages, head // group, slots]
            x = q[rows, head]
            s = (x @ k.T * scale).masked_fill(~seen, -math.inf)
            size = torch.where(seen, x.abs() @ k.abs().T * scale, torch.zeros(()).double()).amax(1, keepdim=True)
            top = s.amax(1, keepdim=True)
            top[~some] = 0
            p = torch.exp(s - top)
            total = p.sum(1, keepdim=True)
            w = p / torch.where(total > 0, total, torch.ones_like(total))
            v0 = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))
            o = torch.stack([w[i][seen[i]] @ v0[seen[i]] if bool(some[i]) else torch.zeros(d).double() for i in range(n)])
            a = torch.stack([w[i][seen[i]] @ v0[seen[i]].abs() if bool(some[i]) else torch.zeros(d).double() for i in range(n)])
            big = torch.stack([v0[seen[i]].abs().amax(0) if bool(some[i]) else torch.zeros(d).double() for i in range(n)])
            out[rows, head] = o
            lse[rows, head] = torch.where(some, (torch.log(total) + top)[:, 0], torch.tensor(-math.inf).double())
            delta = (d + 6) * 2.0 ** -24 * size + 2.0 ** -19
            # the logarithm itself in 32 bits: half a step of the maximum in base 2, of the result, and its own error
            lse_bound[rows, head] = (step * 1.01 + delta[:, 0] + least * seen.sum(1) + 2.0 ** -22 * (top[:, 0].abs() + 12))
            bound[rows, head] = step * o.abs() + (2 * step + 2 * delta) * a + least * (1 + 2 * seen.sum(1, keepdim=True) * big)
    return out, lse, bound, lse_bound

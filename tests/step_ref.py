"""Plain forms of a step with drafted trees, one sequence, token and row after the other: block tables from lengths,
norms of heads, attention over a tree (64 bits), rules on logits, the path taken and the slots it moves to."""
import math

import numpy as np
import torch

import kv_ref
from attention_cuts import Exact


def tree(n, rng, kind="random"):
    """Parents of n nodes, the first without one."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1) if n else []
    return [-1] + [int(rng.integers(max(0, i - 7), i)) for i in range(1, n)] if n else []


def ancestors(parents, i, most=1024):
    """The nodes from i up to one without a parent, i first; nodes from `most` on, and parents that are not before
    their child, are none."""
    got = [i]
    while i < most and 0 <= parents[i] < i:
        i = parents[i]
        got.append(i)
    return got


def mask_rows(parents_by_seq, words):
    """int64 [tokens, words] of lists of parents by sequence."""
    rows = []
    for parents in parents_by_seq:
        for i in range(len(parents)):
            row = [0] * words
            if i < 64 * words:
                for j in ancestors(parents, i):
                    row[j // 64] |= 1 << (j % 64)
            rows.append([x - (1 << 64) if x >> 63 else x for x in row])
    return torch.tensor(rows, dtype=torch.int64).reshape(len(rows), words)


def bits_of(mask, row, n):
    """The j < n whose bits are set in a row."""
    return [j for j in range(min(n, 64 * mask.shape[1])) if (int(mask[row, j // 64]) >> (j % 64)) & 1]


class TreeExact(Exact):
    """Attention over a tree in 64 bits, with the bounds of Exact (the arithmetic is the same; other keys are seen)."""

    def __init__(self, q, k_cache, v_cache, batch, mask, scale, window):
        self.mask = mask
        super().__init__(q, k_cache, v_cache, batch, scale, window)

    def seen(self, b, keys):
        n, c = self.batch.new[b], self.batch.ctx[b]
        past = c - n
        seen = torch.zeros(n, len(keys), dtype=torch.bool)
        for i in range(n):
            on = bits_of(self.mask, int(self.batch.start[b]) + i, n)
            depth = len([j for j in on if j != i])
            cached = keys < past
            if self.window:
                cached &= keys > past + depth - self.window
            seen[i] = cached
            for j in on:
                seen[i] |= keys == past + j
        return seen


def assign(table, held, past, new, free, count, page, tokens, parents=None, words=0):
    """Every output of q4_kv_assign as numpy arrays, rows that are not written as None."""
    seqs, columns = table.shape
    clean = lambda x: np.clip(np.asarray(x, dtype=np.int64), 0, 1 << 30)  # noqa: E731
    past, new = clean(past), clean(new)
    held = np.clip(np.asarray(held, dtype=np.int64), 0, columns)
    count = min(max(int(count), 0), len(free))
    out = dict(table=table.copy(), held=held.copy(), start=[0], ctx=np.minimum(past + new, 2 ** 31 - 1), missing=np.zeros(seqs, np.int64),
               positions=[None] * tokens, slots=[None] * tokens, mask=[None] * tokens)
    left, full = count, False
    for b in range(seqs):
        need = min(-(-int(past[b] + new[b]) // page), columns)
        lack = max(0, need - int(held[b]))
        if lack and (full or lack > left):
            full = True
            out["missing"][b] = lack
            out["table"][b, held[b] : held[b] + lack] = -1
        else:
            for c in range(lack):
                left -= 1
                out["table"][b, held[b] + c] = free[left]
            out["held"][b] += lack
        first = out["start"][-1]
        mine = None if parents is None else [int(parents[first + i]) if first + i < tokens else -1 for i in range(int(new[b]))]
        for i in range(int(new[b])):
            if first + i >= tokens:
                break
            place = int(past[b]) + i
            c = place // page
            got = int(out["table"][b, c]) if c < columns else -1
            out["slots"][first + i] = got * page + place % page if got >= 0 else -1
            most = 64 * words if words else 1024
            if mine is None:
                on, out["positions"][first + i] = range(i + 1), place
            else:
                on = ancestors(mine, i, most)
                out["positions"][first + i] = int(past[b]) + len(on) - 1
                if i >= most:
                    on = []
            row = [0] * words
            for j in on:
                if j < 64 * words:
                    row[j // 64] |= 1 << (j % 64)
            out["mask"][first + i] = [x - (1 << 64) if x >> 63 else x for x in row]
        out["start"].append(first + int(new[b]))
    out["free"] = left
    return out


def norm(x, gain, eps):
    """x [T, H, D] float64 with each head normed."""
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * (1.0 if gain is None else gain.double())


def norm_rope_bound(x, gain, eps, positions, inv_freq, layout, dtype, mscale=1.0):
    """How far the norm and the rotation in 32 bits, rounded once, may be from those in 64.  A lane adds at most 32
    squares in a row and six more sums join the lanes: the mean of squares, all of one sign, is off by at most 40
    2^-24 of itself, its root by half of that, the sum with eps, the root, the division and the two products by one
    rounding each: in all below 26 2^-24 < 2^-19 of each normed element.  The rotation adds what kv_ref.rotate_bound
    says, for elements of that size."""
    y = norm(x, gain, eps)
    size = y.abs().clone()
    r = 0 if inv_freq is None else 2 * len(inv_freq)
    if not r:
        return kv_ref.HALF_STEP[dtype] * (1 + 2.0 ** -18) * y.abs() + kv_ref.LEAST[dtype] + 2.0 ** -19 * size
    first = slice(0, r, 2) if layout == "interleaved" else slice(0, r // 2)
    second = slice(1, r, 2) if layout == "interleaved" else slice(r // 2, r)
    both = (y[..., first].abs() + y[..., second].abs()) * abs(mscale)
    size[..., first], size[..., second] = both, both
    return kv_ref.rotate_bound(y, positions, inv_freq, layout, dtype, mscale) + 2.0 ** -19 * (1 + 2.0 ** -7) * size


class Rules:
    """Rules on logits as host arrays, None where there is none (names of LogitRules)."""

    def __init__(self, seqs, **over):
        self.seqs = seqs
        for name in ("query_start", "history", "history_lens", "prompt_lens", "draft", "mask", "repetition", "presence",
                     "frequency", "bias_start", "bias_tokens", "bias_values", "allowed", "allowed_rows"):
            setattr(self, name, over.get(name))

    def device(self, q4):
        names = [n for n in vars(self) if n != "seqs" and getattr(self, n) is not None]
        return q4.LogitRules(seqs=self.seqs, **{n: torch.as_tensor(getattr(self, n)).cuda() for n in names})

    def rows_of(self, t):
        """The sequence of row t, its first row and its number of rows; None for a row of none."""
        if self.query_start is None:
            return t, t, 1
        for b in range(self.seqs):
            if self.query_start[b] <= t < self.query_start[b + 1]:
                return b, int(self.query_start[b]), int(self.query_start[b + 1] - self.query_start[b])
        return None

    def apply(self, logits, t, kind=np.float32):
        """Row t under the rules, each step rounded to `kind`; None for a row of no sequence."""
        where = self.rows_of(t)
        if where is None:
            return None
        b, first, n = where
        x = np.asarray(logits[t], dtype=np.float32).astype(kind)
        vocab = len(x)
        prompt, answer = [], []
        if self.history is not None:
            text = [int(v) for v in self.history[b][: max(0, min(int(self.history_lens[b]), self.history.shape[1]))]]
            p = max(0, int(self.prompt_lens[b])) if self.prompt_lens is not None else 0
            prompt, answer = text[:p], text[p:]
        if self.draft is not None:
            seen = range(t - first + 1) if self.mask is None else bits_of(self.mask, t, n)
            answer = answer + [int(self.draft[first + j]) for j in seen]
        count = np.zeros(vocab, dtype=np.int64)
        for v in answer:
            if 0 <= v < vocab:
                count[v] += 1
        seen = count > 0
        for v in prompt:
            if 0 <= v < vocab:
                seen[v] = True
        with np.errstate(all="ignore"):
            if self.repetition is not None:
                r = kind(self.repetition[b])
                x = np.where(seen, np.where(x > 0, x / r, x * r), x).astype(kind)
            if self.frequency is not None:
                x = np.where(seen, x - kind(self.frequency[b]) * count.astype(kind), x).astype(kind)
            if self.presence is not None:
                x = np.where(count > 0, x - kind(self.presence[b]), x).astype(kind)
            if self.bias_start is not None:
                last = {}
                for i in range(int(self.bias_start[b]), int(self.bias_start[b + 1])):
                    last[int(self.bias_tokens[i])] = kind(self.bias_values[i])
                for v, value in last.items():
                    if 0 <= v < vocab:
                        x[v] = x[v] + value
        if self.allowed is not None:
            r = t if self.allowed_rows is None else int(self.allowed_rows[t])
            if 0 <= r < len(self.allowed):
                words = np.asarray(self.allowed[r]).astype(np.int64) & 0xFFFFFFFF
                bit = (words[np.arange(vocab) // 32] >> (np.arange(vocab) % 32)) & 1
                x = np.where(bit == 1, x, kind(-math.inf))
        return x

    @staticmethod
    def pick(x):
        y = np.where(np.isnan(x), -math.inf, x)
        return int(np.argmax(y)) if y.max() > -math.inf else -1


def accept(start, ctx, choice, draft, parents, tokens, history=None):
    """accepted, next, path, lens as lists (and the history written)."""
    accepted, following, lens = [], [], []
    path = [None] * tokens
    for b in range(len(ctx)):
        first, last = int(start[b]), int(start[b + 1])
        n = 0 if first < 0 or last > tokens or last < first else last - first
        past = int(ctx[b]) - max(last - first, 0)
        got = [0] if n else []
        while got:
            cur = got[-1]
            want = int(choice[first + cur])
            after = [i for i in range(cur + 1, n)
                     if (i - 1 if parents is None else int(parents[first + i])) == cur and int(draft[first + i]) == want and want >= 0]
            if not after:
                break
            got.append(after[0])
        for j in range(n):
            path[first + j] = got[j] if j < len(got) else -1
        if history is not None:
            for j, i in enumerate(got):
                if 0 <= past + j < history.shape[1]:
                    history[b, past + j] = draft[first + i]
        accepted.append(len(got))
        following.append(int(choice[first + got[-1]]) if got else -1)
        lens.append(past + len(got))
    return accepted, following, path, lens


def move(cache, table, page, pages, start, ctx, path, accepted):
    """A cache [pages, heads, page, dim] with the paths' slots moved, all read before any is written."""
    out = cache.clone()

    def place(b, p):
        if p < 0 or p // page >= table.shape[1] or not 0 <= int(table[b, p // page]) < pages:
            return None
        return int(table[b, p // page]), p % page

    for b in range(len(ctx)):
        n = int(start[b + 1] - start[b])
        past = int(ctx[b]) - n
        for j in range(min(int(accepted[b]), n)):
            node = int(path[int(start[b]) + j])
            if not j < node < n:
                continue
            source, target = place(b, past + node), place(b, past + j)
            if source and target:
                out[target[0], :, target[1]] = cache[source[0], :, source[1]]
    return out

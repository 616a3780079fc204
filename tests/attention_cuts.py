"""Calls of attention that reach every kernel by construction: items of 16, 32, 64 and 128 rows, taken whole and cut
into parts, for every head_dim, with and without a window; and how the library would cut a call."""
import ctypes
import os
import subprocess

import torch

import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "q4_dequant_gemv_block_amd", "csrc")

# new tokens and contexts, query heads (of 2 kv heads): most rows of a kv head 15, 30 and 300
FEW = ([(3, 700), (1, 333), (0, 90), (5, 5), (2, 1100), (1, 0)], 6)
SOME = ([(6, 700), (1, 333), (0, 0), (4, 3), (5, 1100)], 10)
MANY = ([(70, 700), (1, 65), (0, 17), (150, 260), (40, 38)], 4)
FAR = ([(70, 6500), (1, 65), (150, 2700), (40, 38)], 4)
# with and without a window, cut and whole: sequences, window, rows behind the last sequence, and the longest context
# that the call names, right or not: they decide how it is cut
CHOICE = {
    (16, True): ((FEW, 0, 3, 300), (FEW, 100, 3, 300)), (16, False): ((FEW, 0, 3, 60000), (FEW, 300, 6000, 60000)),
    (32, True): ((SOME, 0, 3, 300), (SOME, 100, 3, 300)), (32, False): ((SOME, 0, 3, 60000), (SOME, 300, 6000, 60000)),
    (64, True): ((MANY, 0, 3, 300), (MANY, 100, 3, 300)), (64, False): ((MANY, 0, 3, 3000), (FAR, 2500, 3, 60000)),
    (128, True): ((MANY, 0, 20000, 700), (MANY, 100, 20000, 700)), (128, False): ((MANY, 0, 3, 60000), (FAR, 6000, 1500, 60000)),
}


class Case:
    """rows of an item, head_dim, whole or cut, and what makes it so; pages of several sizes."""

    def __init__(self, rows, dim, whole, windowed, page):
        (self.lens, self.hq), self.window, self.pad, self.max_context = CHOICE[rows, whole][windowed]
        self.rows, self.dim, self.whole, self.page, self.hk = rows, dim, whole, page, 2
        self.max_query = max(n for n, _ in self.lens)
        self.columns = -(-max(self.max_context, max(c for _, c in self.lens)) // page)

    def __repr__(self):
        return "%d rows of %d, %s, window %d, pages of %d" % (self.rows, self.dim, "whole" if self.whole else "cut", self.window, self.page)

    def batch(self, seed):
        return kv_ref.Batch(self.lens, self.page, seed=seed, pad_rows=self.pad, columns=self.columns)


def cases():
    pages = [8, 24, 32, 64, 16, 128, 40]
    got = []
    for dim in (64, 96, 128, 256):
        for rows, whole in CHOICE:
            for windowed in (False, True):
                got.append(Case(rows, dim, whole, windowed, pages[len(got) % len(pages)]))
    return got


def shim(folder):
    """The library's rule for cutting calls, compiled by itself for the host."""
    src, lib = os.path.join(folder, "shape.cpp"), os.path.join(folder, "shape.so")
    with open(src, "w") as f:
        f.write('''#include "attn_shape.h"
extern "C" void shape(int page, int hk, int dim, int columns, int seqs, int hq, long long tokens, int window, int max_query,
                      int max_context, int* rows, int* whole) {
    q4::CacheArg c = {};
    c.page_size = q4::FastDiv(page);
    c.kv_heads = hk;
    c.head_dim = dim;
    q4::BatchArg b = {};
    b.table_pages = columns;
    b.seqs = seqs;
    const q4::AttnShape s = q4::attn_shape_on(256, c, b, hq, tokens, window, max_query, max_context);
    *rows = s.rows;
    *whole = s.bytes == 0;
}
''')
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                           "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), src, "-o", lib])
    fn = ctypes.CDLL(lib).shape
    fn.argtypes = [ctypes.c_int] * 6 + [ctypes.c_longlong] + [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)] * 2

    def shape(case):
        rows, whole = ctypes.c_int(), ctypes.c_int()
        tokens = sum(n for n, _ in case.lens) + case.pad
        fn(case.page, case.hk, case.dim, case.columns, len(case.lens), case.hq, tokens, case.window, case.max_query,
           case.max_context, rows, whole)
        return rows.value, bool(whole.value)
    return shape


class Exact:
    """The same attention in 64 bits, each sequence's keys side by side, with the bounds of kv_ref.attention (their
    derivation is there)."""

    def __init__(self, q, k_cache, v_cache, batch, scale, window):
        t, h, d = q.shape
        hk = k_cache.shape[1]
        step, least = kv_ref.HALF_STEP[q.dtype], kv_ref.LEAST[q.dtype]
        self.batch, self.window, self.group = batch, window, h // hk
        self.out = torch.zeros(t, h, d, dtype=torch.float64)
        self.lse = torch.full((t, h), -float("inf"), dtype=torch.float64)
        self.bound = torch.full((t, h, d), least, dtype=torch.float64)
        self.lse_bound = torch.zeros(t, h, dtype=torch.float64)
        self.weights = {}
        for b in range(len(batch.new)):
            places = batch.places(b)
            n, c = batch.new[b], batch.ctx[b]
            if not n or not places:
                continue
            rows = slice(int(batch.start[b]), int(batch.start[b + 1]))
            pages, slots = torch.tensor([x for _, x, _ in places]), torch.tensor([s for _, _, s in places])
            k = k_cache[pages, :, slots].double().transpose(0, 1).repeat_interleave(self.group, 0)  # heads, keys, dim
            v = v_cache[pages, :, slots].double().transpose(0, 1).repeat_interleave(self.group, 0)
            x = q[rows].double().transpose(0, 1)
            seen = self.seen(b, torch.tensor([p for p, _, _ in places]))
            some = seen.any(1)
            s = (torch.matmul(x, k.transpose(1, 2)) * scale).masked_fill(~seen, -float("inf"))
            size = (torch.matmul(x.abs(), k.abs().transpose(1, 2)) * scale).masked_fill(~seen, 0).amax(2, keepdim=True)
            top = s.amax(2, keepdim=True)
            top[:, ~some] = 0
            p = torch.exp(s - top)
            total = p.sum(2, keepdim=True)
            w = p / torch.where(total > 0, total, torch.ones_like(total))
            self.weights[b] = w
            o, a = torch.matmul(w, v), torch.matmul(w, v.abs())
            big = torch.stack([v[:, :, e].abs().unsqueeze(1).masked_fill(~seen, 0).amax(2) for e in range(d)], 2)
            count = seen.sum(1)[None, :, None]
            delta = (d + 6) * 2.0 ** -24 * size + 2.0 ** -19
            self.out[rows] = o.transpose(0, 1)
            lse = torch.where(some[None, :], (torch.log(total) + top)[..., 0], torch.tensor(-float("inf")).double())
            self.lse[rows] = lse.transpose(0, 1)
            self.lse_bound[rows] = (step * 1.01 + delta[..., 0] + least * count[..., 0] + 2.0 ** -22 * (top[..., 0].abs() + 12)).transpose(0, 1)
            self.bound[rows] = (step * o.abs() + (2 * step + 2 * delta) * a + least * (1 + 2 * count * big)).transpose(0, 1)

    def seen(self, b, keys):
        """Which of these positions each new token of a sequence sees."""
        n, c = self.batch.new[b], self.batch.ctx[b]
        at = torch.arange(c - n, c)[:, None]
        seen = keys[None, :] <= at
        return seen & (keys[None, :] > at - self.window) if self.window else seen

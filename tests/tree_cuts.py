"""Calls of attention over trees that reach every kernel by construction: items of 16 to 256 rows, taken whole and cut into
parts, for every head_dim, with and without a window; and how the library would cut a call."""
import ctypes
import os
import subprocess

import attention_cuts
import kv_ref

# new tokens and contexts; query heads of 2 kv heads
ONE = [(3, 700), (1, 333), (0, 90), (5, 5), (2, 1100), (1, 0)]  # at most 15 rows
TWO = [(6, 700), (1, 333), (0, 0), (4, 3), (5, 1100)]           # 30
SOME = [(20, 700), (9, 64), (0, 9), (31, 40), (7, 1000)]        # 62 or 124
MANY = [(70, 700), (1, 65), (0, 17), (150, 260), (40, 38)]      # 300
WIDE = [(50, 700), (1, 65), (0, 17), (64, 260), (40, 38)]       # 192
FAR = [(50, 6500), (1, 65), (64, 2700), (40, 38)]
NEAR = [(30, 700), (1, 65), (0, 17), (32, 260), (20, 38)]       # 128 of 8 heads
NEARFAR = [(32, 6500), (1, 65), (30, 2700), (20, 38)]
FARTHER = [(50, 17000), (64, 2700), (40, 38)] + [(0, 9)] * 9
# rows of an item, whole -> sequences, query heads, window, rows behind the last sequence, the longest context that the
# call names, right or not, without and with a window: they decide how it is cut
CHOICE = {
    (16, True): ((ONE, 6, 0, 3, 300), (ONE, 6, 100, 3, 300)), (16, False): ((ONE, 6, 0, 3, 60000), (ONE, 6, 30000, 3, 60000)),
    (32, True): ((TWO, 10, 0, 3, 300), (SOME, 4, 100, 3, 300)), (32, False): ((TWO, 10, 0, 3, 60000), (TWO, 10, 6000, 6000, 60000)),
    (64, True): ((MANY, 4, 0, 3, 300), (MANY, 4, 100, 3, 300)), (64, False): ((MANY, 4, 0, 3, 3000), (FAR, 8, 2500, 3, 60000)),
    (128, True): ((MANY, 4, 0, 90000, 700), (MANY, 4, 100, 90000, 700)), (128, False): ((MANY, 4, 0, 3, 60000), (FAR, 8, 2500, 1200, 6500)),
    (256, False): ((WIDE, 6, 0, 300, 60000), (FARTHER, 6, 16000, 3000, 32000)),
}
# heads that items of 256 rows are for: those of 128 have parts where no sequence has more rows
NARROW = ((NEAR, 8, 0, 300, 60000), (NEARFAR, 8, 4000, 2000, 6500))


class Case:
    """rows of an item, head_dim, whole or cut, and what makes it so; pages of several sizes."""

    def __init__(self, rows, dim, whole, windowed, page):
        choice = NARROW if (rows, whole) == (128, False) and dim in (96, 128) else CHOICE[rows, whole]
        self.lens, self.hq, self.window, self.pad, self.max_context = choice[windowed]
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
                if rows < 256 or dim in (96, 128):
                    got.append(Case(rows, dim, whole, windowed, pages[len(got) % len(pages)]))
    return got


def shim(folder):
    """The library's rule for cutting calls over trees, compiled by itself for the host: (rows of an item, whole)."""
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
    const q4::AttnShape s = q4::attn_shape_on(256, c, b, hq, tokens, window, max_query, max_context, true);
    *rows = s.rows;
    *whole = s.bytes == 0;
}
''')
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                           "-I" + attention_cuts.CSRC, "-I" + os.path.join(attention_cuts.ROOT, "include"), src, "-o", lib])
    fn = ctypes.CDLL(lib).shape
    fn.argtypes = [ctypes.c_int] * 6 + [ctypes.c_longlong] + [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int)] * 2

    def shape(case):
        rows, whole = ctypes.c_int(), ctypes.c_int()
        tokens = sum(n for n, _ in case.lens) + case.pad
        fn(case.page, case.hk, case.dim, case.columns, len(case.lens), case.hq, tokens, case.window, case.max_query,
           case.max_context, rows, whole)
        return rows.value, bool(whole.value)
    return shape

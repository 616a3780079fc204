// How a call of attention is cut: a rule on sizes, on the host alone.
#pragma once

#include "kv_launch.h"

#include <algorithm>
#include <cmath>

namespace q4 {

constexpr int kAttnStep = 32;  // keys a wave of k_attn takes at a time

// Places for the items of a call, the most that it can have: the rows of a sequence
// with new tokens round up once, or those of each token; and whether it is the
// second (Places in attn_device.h).
inline int64_t item_bound(const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int rows, int* per_token) {
    const int group = q_heads / c.kv_heads, each = (group + rows - 1) / rows;
    const int64_t by_rows = tokens * group / rows + std::min<int64_t>(b.seqs, tokens);
    *per_token = tokens * each <= by_rows ? each : 0;
    return c.kv_heads * (*per_token ? tokens * each : by_rows);
}

// Trees have few rows over long contexts, their tiles wait less (attn_tile.h) and
// their parts are joined by item, so they have numbers of their own, and more ways:
// up to 128 rows in items of 32 (many workgroups of little each: 16 tokens of 4 heads
// a kv head over 515 keys 11.7 us, in one item of 64 rows 14.9), more than 128 of heads
// of 96 or 128 in items of 256, whose halves two workgroups of one XCD have at a time:
// the keys come from HBM once (3 sequences of 64 tokens over 32768 keys, 32/8 heads of
// 128, f16, 139 us, with items of 128 161; of 40 tokens over 6000 keys 43 and 52).
// The numbers for heads up to 128 are fitted to 378 calls.  Of 1044 (2 to 200 tokens of 1
// to 96 sequences over up to 40000 keys, heads of 64 to 256, with and without windows),
// each run in every way, what is taken is 1.3 % behind the best in the mean, within 5 %
// of it in 959 and 28 % behind at most.
struct TreeCost {
    double start, each;     // us of an item, of 256 keys (items of 16 and 32 rows) or a tile
    double alone, late;     // a whole item on a CU of its own; of what the last round lacks
    double parts, range, traffic;  // the join's launch, units in ranges, the parts' way to memory and back
};
inline TreeCost tree_cost(int rows, int head_dim) {
    const double dim = head_dim / 128.0;
    if (rows <= 32) return {1.4, (0.213 + 2.18 * dim) * (rows == 32 ? 1.05 : 1.0), 1.0, 1.24, 10.4, 1.0, 0.71};
    if (head_dim > 128) return {0.38, rows == 64 ? 1.82 : 2.14, 0.95, 0.16, 10.1, 1.17, 0.87};
    const double tile = rows == 64 ? 0.431 + 0.617 * dim : (0.422 + 0.738 * dim) * (rows == 256 ? 0.711 : 1.0);
    return {0.533, tile, 0.906, 0.166, 9.65, 1.302, 0.921};
}

// Workgroups that the machine holds at a time, and the workspace of as many with parts.
inline int attn_slots(int cus, int rows, int head_dim) { return rows <= 32 || rows == 256 || head_dim > 128 ? cus : 2 * cus; }
inline size_t attn_parts_bytes(int grid, int rows, int head_dim) {
    return (size_t)2 * grid * rows * (head_dim * sizeof(float) + 2 * sizeof(float));
}
inline bool attn_rows_256(int head_dim) { return head_dim == 96 || head_dim == 128; }  // items of 256 rows, of trees

// The most that a call with up to `most` query rows of a kv head takes.  (One call's need
// is not such a bound: fewer rows or keys may be cut where more are taken whole, and into
// larger items.)
inline size_t attn_workspace_most(int cus, int head_dim, int64_t most) {
    size_t bytes = 0;
    auto consider = [&](int rows, bool taken) {
        if (taken) bytes = std::max(bytes, attn_parts_bytes(attn_slots(cus, rows, head_dim), rows, head_dim));
    };
    consider(16, true);
    consider(32, most > 16);
    consider(64, most > 32);
    consider(128, most > 32);
    consider(256, most > 128 && attn_rows_256(head_dim));
    return bytes;
}

// How a call is cut: the rows of an item, and whether items are taken whole or
// in parts.  Parts cost a launch that waits for the first one (measured 5 to 7
// us), their way to memory and back at about 4 TB/s, and in tiles the L2: whole
// items of one kv head run side by side and read the same keys, ranges do not.
// Whole items cost what the longest of them takes alone.  Both are estimated
// from the longest context and the most new tokens of a sequence, as far as the
// caller knows them, and the cheapest way is taken.
//
// The estimates are numbers to compare ways by, of the size of microseconds but no
// forecast (a windowed call of 34 us is put at 18, a chunk of 490 at 385).  They are
// fits to calls run in each way, head_dim 64 to 256, equal and ragged, with and
// without windows, made when whole items took up to 1.5 us longer to start.  As the
// kernels are now: tiles, 560 calls of 64 to 4096 new tokens of 1 to 30 sequences, up
// to 30000 keys: what is taken is within 5 % of the best of the four ways in 524 and
// 19 % behind at most.  k_attn, 264 calls of 1 to 4 new tokens of 1 to 200 sequences,
// up to 20000 keys: 251 within 5 % of the better way, 38 % behind at most; of 96
// batches of 16 to 200 sequences, half of them with lengths from 1/16 of the longest
// up, which the host cannot see, 80, and 64 % behind at most (many short items of a
// range, each of which starts with nothing on its way).
inline AttnShape attn_shape_on(int cus, const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int window, int max_query, int max_context, bool tree = false) {
    const int64_t group = q_heads / c.kv_heads, capacity = (int64_t)b.table_pages * c.page_size.d;
    const int64_t longest = max_query > 0 ? std::min<int64_t>(max_query, tokens) : tokens;  // new tokens of a sequence
    const int64_t most = longest * group;
    const int64_t seqs = std::min<int64_t>(b.seqs, tokens);
    const int64_t context = max_context > 0 ? std::min<int64_t>(max_context, capacity) : capacity;
    const double dim = c.head_dim / 128.0;
    AttnShape best = {};
    double best_cost = 0;
    auto consider = [&](int rows) {
        AttnShape s = {};
        s.rows = rows;
        s.step = rows <= 32 ? kAttnStep : 64;
        s.unit = 64;
        s.most_rows = (int)std::min<int64_t>(rows, most);
        const int slots = attn_slots(cus, rows, c.head_dim);
        // keys of an item, the part of them that its sequence's items see on average, and all items
        const int64_t keys = window ? std::min<int64_t>(context, (int64_t)window + (tree ? longest : (rows - 1) / group) + 2) : context;
        const int64_t past = std::max<int64_t>(context - longest, 0);
        const double inside = (double)std::min(std::max<int64_t>(keys - past, 0), longest);  // tokens that see less
        const double seen = std::min(1.0, (inside * past + inside * (inside + 1) / 2 + (longest - inside) * keys) / ((double)longest * keys));
        const double items = (double)c.kv_heads * (longest * seqs == tokens ? seqs * ((most + rows - 1) / rows) : (tokens * group + rows * seqs / 2) / rows);
        const double rounds = items / slots, work = seen * rounds;
        const double late = std::min(1.0, std::ceil(rounds) - work);  // what the last round lacks
        const double parts = std::min<double>(slots, items * keys / s.unit);
        const double traffic = parts * s.most_rows * c.head_dim * 8 / 4e6;
        double whole, cut;
        if (tree) {
            const TreeCost cost = tree_cost(rows, c.head_dim);
            const double us = cost.each * (rows <= 32 ? keys / 256.0 : (double)((keys + 63) / 64));
            whole = rows <= 32 ? cost.start + us * (rounds > 1 ? rounds + cost.late * std::min(1.0, std::ceil(rounds) - rounds) : 1.0)
                    : items <= cus ? cost.alone * (cost.start + us)
                                   : cost.start + us * std::max(1.0, rounds + cost.late * std::min(1.0, std::ceil(rounds) - rounds));
            cut = cost.parts + cost.range * us * rounds + cost.traffic * traffic;
        } else if (rows <= 32) {
            const double us = keys / 256.0 * (0.25 + 1.85 * dim);  // an item's steps
            whole = (1.3 + us) * (rounds > 1 ? work + 1.2 * late : 1.0);
            cut = us * rounds * (c.head_dim == 64 ? 1.4 : 1.0) + 6 + traffic;  // two whole items of 64 share a CU
        } else {
            const double tiles = (double)((keys + 63) / 64);
            const double shared = 0.55 + tiles * (c.head_dim > 128 ? (rows == 64 ? 2.25 : 2.8) : rows == 64 ? 0.4 + 0.75 * dim : 0.5 + dim);
            const double alone = c.head_dim > 128 ? shared : shared * (rows == 64 ? 0.75 : 0.8);  // on its CU
            whole = items <= cus ? alone : rounds <= 1 ? shared : shared * std::max(1.0, work + 0.65 * late);
            cut = 1.15 * shared * rounds * (0.85 + 0.15 * seen) + 15 + traffic;
        }
        const int64_t bound = item_bound(c, b, q_heads, tokens, rows, &s.per_token);
        if (whole <= cut && bound < (int64_t(1) << 31) && rows <= 128) {
            s.unit = 1 << 30;
            s.places = (int)bound;
        } else {
            // larger units where this many would pass 31 bits
            while (s.unit < (1 << 30) && bound * (capacity / s.unit + 1) >= (int64_t(1) << 31)) s.unit *= 2;
            s.grid = slots;
            s.few = items * 8 <= slots;
            s.bytes = attn_parts_bytes(s.grid, s.rows, c.head_dim);
        }
        const double taken = rows <= 128 ? std::min(whole, cut) : cut;  // items of 256 are not taken whole
        if (!best.rows || taken < best_cost) {
            best = s;
            best_cost = taken;
        }
    };
    if (most <= 32) {
        consider(most <= 16 ? 16 : 32);
    } else {
        if (tree && most <= 128) consider(32);
        consider(64);
        consider(128);
        if (tree && most > 128 && attn_rows_256(c.head_dim)) consider(256);
    }
    return best;
}

}  // namespace q4

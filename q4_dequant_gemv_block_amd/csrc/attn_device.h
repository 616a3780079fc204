// Device-side parts shared by the attention kernels: how a call's work is cut
// into items, units and ranges, and where parts of an item are kept.
#pragma once

#include "kv_device.h"

#include <atomic>
#include <type_traits>

namespace q4 {

// Allows a kernel more than 64 KiB of LDS, once a device.
struct LdsLimit {
    std::atomic<bool> done[64];
    hipError_t raise(const void* kernel, size_t bytes);
};

struct Cut;
// The kernel for many query rows of a sequence (attn_tile.hip).
template <typename T, int D>
hipError_t launch_attn_tile(const AttnArgs& a, const Cut& cut, const AttnShape& shape, hipStream_t s);

// log2 by which a score may exceed the running maximum before that is raised:
// probabilities stay below 2^8, far inside both types.
constexpr float kRaise = 8.0f;
constexpr float kNone = -__builtin_inff();

// Two floats rounded to T in one dword (first in the low half), and back.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef typename T::elem e2 __attribute__((ext_vector_type(2)));
    const e2 v = {(typename T::elem)a, (typename T::elem)b};
    return __builtin_bit_cast(uint32_t, v);
}
template <typename T>
__device__ __forceinline__ float unpack_sum(uint32_t v) {
    typedef typename T::elem e2 __attribute__((ext_vector_type(2)));
    const e2 x = __builtin_bit_cast(e2, v);
    return (float)x[0] + (float)x[1];
}

// The halves of a dword that hold NaN or an infinity, as a mask.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite(uint32_t v) {
    constexpr uint32_t e = std::is_same<T, F16>::value ? 0x7C00u : 0x7F80u;
    return ((v & e) == e ? 0xFFFFu : 0u) | ((v & (e << 16)) == (e << 16) ? 0xFFFF0000u : 0u);
}
template <typename T>
__device__ __forceinline__ float half_of(uint32_t v, int high) {
    const uint16_t h = (uint16_t)(high ? v >> 16 : v);
    return (float)__builtin_bit_cast(typename T::elem, h);
}

// Orders a wave's own LDS accesses (which the hardware runs in order).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// What one sequence asks for.
struct Seq {
    int b, row0, n, ctx;  // first row, new tokens, context
    int tiles, units;     // items of a kv head, units of an item
};

struct Cut {
    int rows, unit, step, group, window, kv_heads, capacity;  // an item's keys begin at a multiple of step
    int64_t tokens;
};

// n new tokens with the given context: items of a kv head and units of an item
// (the most that any of its items has; a unit that lies behind an item's last
// visible key holds no work).
__device__ __forceinline__ void cut_sequence(const Cut& c, const BatchArg& batch, int b, Seq* s) {
    const int first = batch.query_start[b], last = batch.query_start[b + 1];
    s->b = b;
    s->row0 = first;
    s->ctx = batch.context_len[b];
    s->n = first < 0 || last > c.tokens || last < first ? 0 : last - first;
    const int keys = max(0, min(s->ctx, c.capacity));
    int span = keys;
    if (c.window) {
        const int64_t most = (int64_t)c.window + (c.rows - 1) / c.group + 1 + c.step;
        span = (int)min((int64_t)keys, most);
    }
    s->tiles = (int)(((int64_t)s->n * c.group + c.rows - 1) / c.rows);
    s->units = s->n ? max(1, (span + c.unit - 1) / c.unit) : 0;
}

__device__ __forceinline__ uint32_t seq_units(const Cut& c, const BatchArg& batch, int b) {
    if (b >= batch.seqs) return 0;
    Seq s;
    cut_sequence(c, batch, b, &s);
    return (uint32_t)c.kv_heads * s.tiles * s.units;
}

__device__ __forceinline__ uint32_t wave_sum_u32(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += (uint32_t)__shfl_xor((int)v, o);
    return v;
}

// The sequence that holds unit `at`, and the first unit of that sequence; by
// whole waves, 64 sequences at a time.
__device__ __forceinline__ int find_unit(const Cut& c, const BatchArg& batch, uint32_t at, uint32_t* begin) {
    const int lane = threadIdx.x & 63;
    uint32_t base = 0;
    for (int b0 = 0; b0 < batch.seqs; b0 += 64) {
        const uint32_t u = seq_units(c, batch, b0 + lane);
        uint32_t incl = u;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t t = (uint32_t)__shfl_up((int)incl, o);
            if (lane >= o) incl += t;
        }
        const uint64_t past = __ballot(base + incl > at);
        if (past) {
            const int l = __builtin_ctzll(past);
            *begin = base + (uint32_t)__shfl((int)(incl - u), l);
            return b0 + l;
        }
        base += (uint32_t)__shfl((int)incl, 63);
    }
    *begin = base;
    return -1;
}

__device__ __forceinline__ uint32_t all_units(const Cut& c, const BatchArg& batch) {
    uint32_t sum = 0;
    for (int b0 = 0; b0 < batch.seqs; b0 += 64) sum += seq_units(c, batch, b0 + (int)(threadIdx.x & 63));
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)wave_sum_u32(sum));
}

// First unit of workgroup w's range.
__device__ __forceinline__ uint32_t range_begin(uint32_t total, uint32_t w, uint32_t grid) {
    return (uint32_t)((uint64_t)total * w / grid);
}

// One item's keys, or a part of them, as a workgroup gets them.
struct Item {
    int u0, u1;           // units of the item, of seq.units
    int head, row0, rows; // kv head, first query row of the sequence, query rows
    int past;             // position of the sequence's first new token
    int p_first, p_last;  // positions of the first and the last row
    int k_lo, k_hi;       // keys of the part
};

// Items of a sequence in order: the last rows first (they see most keys, and
// what takes longest should start first), their kv heads side by side (with 8
// XCDs taking workgroups in turn, an XCD's L2 then sees few heads).
__device__ __forceinline__ void place_item(const Cut& c, const Seq& seq, uint32_t item, Item* x) {
    const int tile = seq.tiles - 1 - (int)(item / (uint32_t)c.kv_heads);
    x->head = (int)(item % (uint32_t)c.kv_heads);
    x->row0 = tile * c.rows;
    x->rows = min(c.rows, seq.n * c.group - x->row0);
}

// The items of workgroup blockIdx.x's range.
struct Work {
    uint32_t lo, hi, begin;
    Seq seq;

    __device__ __forceinline__ bool start(const Cut& c, const BatchArg& batch) {
        const uint32_t total = all_units(c, batch), grid = min((uint32_t)gridDim.x, total);  // no range is empty
        if (blockIdx.x >= grid) return false;
        lo = range_begin(total, blockIdx.x, grid);
        hi = range_begin(total, blockIdx.x + 1, grid);
        uint32_t first;
        const int b = __builtin_amdgcn_readfirstlane(find_unit(c, batch, lo, &first));
        begin = (uint32_t)__builtin_amdgcn_readfirstlane((int)first);
        if (b < 0) return false;
        cut_sequence(c, batch, b, &seq);
        return true;
    }

    __device__ __forceinline__ bool next(const Cut& c, const BatchArg& batch, Item* x) {
        if (lo >= hi) return false;
        while (lo - begin >= (uint32_t)c.kv_heads * seq.tiles * seq.units) {
            begin += (uint32_t)c.kv_heads * seq.tiles * seq.units;
            if (seq.b + 1 >= batch.seqs) return false;
            cut_sequence(c, batch, seq.b + 1, &seq);
        }
        const uint32_t item = (lo - begin) / (uint32_t)seq.units;
        x->u0 = (int)((lo - begin) - item * seq.units);
        x->u1 = (int)min((uint32_t)seq.units, x->u0 + (hi - lo));
        lo += x->u1 - x->u0;
        place_item(c, seq, item, x);
        x->past = seq.ctx - seq.n;
        x->p_first = x->past + x->row0 / c.group;
        x->p_last = x->past + (x->row0 + x->rows - 1) / c.group;
        const int keys = max(0, min(min(seq.ctx, c.capacity), x->p_last + 1));
        const int start = c.window ? max(0, x->p_first - c.window + 1) / c.step * c.step : 0;
        x->k_lo = (int)min((int64_t)keys, start + (int64_t)x->u0 * c.unit);
        x->k_hi = (int)min((int64_t)keys, start + (int64_t)x->u1 * c.unit);
        return true;
    }
};

// Parts in the workspace: every workgroup has at most two, one that begins its
// range (slot 0) and one whose item begins inside it and ends behind it (slot 1).
template <int D>
struct Parts {
    float* o;   // [2 grid][rows][D]
    f2* ml;     // [2 grid][rows]: maximum (log2), sum
    int rows;
    __device__ Parts(void* ws, int grid, int rows_) : rows(rows_) {
        o = static_cast<float*>(ws);
        ml = reinterpret_cast<f2*>(o + (int64_t)2 * grid * rows_ * D);
    }
};

// 1 / sum of a row's weights, 0 for a row that sees no key (NaN stays NaN).
__device__ __forceinline__ float row_scale(float sum) { return sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f; }
// The natural log of 2^top * sum.
__device__ __forceinline__ float row_lse(float top, float sum) {
    return sum > 0.0f ? (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f : (sum != sum ? sum : kNone);
}

}  // namespace q4

// Device-side parts shared by the attention kernels: how a call's work is cut
// into items, units and ranges, and where parts of an item are kept.
#pragma once

#include "kv_device.h"

#include <algorithm>
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

// A row's weights are 2^(score - m).  m is set to kLift below the largest score, and
// set anew when a score exceeds it by kRaise (each 2^8 of scores at the soonest).
// In binary16 the largest weight is then between 2^7 and 2^15, so that weights keep
// their 11 bits down to 2^-21 of it and come to 0 at 2^-32 (from 2^0 they would at
// 2^-25, a part of the sum that counts where there are 10^5 of them).  bfloat16 has
// the exponents: 2^0 to 2^8.
template <typename T>
constexpr float kLift = std::is_same<T, F16>::value ? 7.0f : 0.0f;
template <typename T>
constexpr float kRaise = kLift<T> + 8.0f;
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

// Bits 15 and 31: the halves of a dword that hold NaN or an infinity (an
// exponent of ones carries into the sign's place), and those halves as a mask.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t v) {
    constexpr uint32_t e = std::is_same<T, F16>::value ? 0x7C007C00u : 0x7F807F80u;
    constexpr uint32_t one = std::is_same<T, F16>::value ? 0x04000400u : 0x00800080u;
    return ((v & e) + one) & 0x80008000u;
}
template <typename T>
__device__ __forceinline__ uint32_t nonfinite(uint32_t v) {
    const uint32_t b = nonfinite_bits<T>(v);
    return (b << 1) - (b >> 15);
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

// How a call is cut (AttnShape with its numbers as shifts and products).
struct Cut {
    int rows_log2, unit_log2, step;  // an item's keys begin at a multiple of step
    int window, capacity;            // capacity: tokens a row of the block table holds
    uint32_t place;                  // items taken whole (Places): the first workgroup's place
    int per_token;                   // places of a token and kv head; 0: by rows
    FastDiv group, kv_heads;
    int64_t tokens;
};

// Launches a call's workgroups with what they are told: those of whole items 2^22 at
// a time (a launch has fewer than 2^32 threads along an axis).
template <typename L>
hipError_t launch_shape(const AttnShape& shape, Cut cut, L launch) {
    if (!shape.places) launch((unsigned)shape.grid, cut);
    for (int64_t at = 0; at < shape.places; at += 1 << 22) {
        cut.place = (uint32_t)at;
        launch((unsigned)std::min<int64_t>(shape.places - at, 1 << 22), cut);
    }
    return hipGetLastError();
}

// What one sequence asks for.
struct Seq {
    int b, row0, n, ctx;  // first row, new tokens, context
    int tiles, units;     // items of a kv head, units of an item
};

// Items of a kv head and units of an item (the most that any of the sequence's
// items has: a unit behind an item's last visible key holds no work).
__device__ __forceinline__ void cut_sequence(const Cut& c, Seq* s) {
    int span = max(0, min(s->ctx, c.capacity));
    if (c.window) {
        const int64_t most = (int64_t)c.window + (int)c.group.div((1u << c.rows_log2) - 1) + 1 + c.step;
        span = (int)min((int64_t)span, most);
    }
    s->tiles = (int)(((int64_t)s->n * c.group.d + (1 << c.rows_log2) - 1) >> c.rows_log2);
    s->units = s->n ? max(1, (int)(((int64_t)span + (1 << c.unit_log2) - 1) >> c.unit_log2)) : 0;
}

// Sequence b.  One whose rows are not all among the call's has no new tokens.
__device__ __forceinline__ void read_sequence(const Cut& c, const BatchArg& batch, int b, Seq* s) {
    const int first = batch.query_start[b], last = batch.query_start[b + 1];
    s->b = b;
    s->ctx = batch.context_len[b];
    s->row0 = first;
    s->n = first < 0 || last > c.tokens || last < first ? 0 : last - first;
}

// First unit of range w of `grid`.
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
    const int up = (int)c.kv_heads.div(item);
    x->head = (int)item - up * (int)c.kv_heads.d;
    x->row0 = (seq.tiles - 1 - up) << c.rows_log2;
    x->rows = min(1 << c.rows_log2, seq.n * (int)c.group.d - x->row0);
}

// Positions of an item's rows and the keys of its units [u0, u1).
__device__ __forceinline__ void place_keys(const Cut& c, const Seq& seq, Item* x) {
    x->past = seq.ctx - seq.n;
    x->p_first = x->past + (int)c.group.div(x->row0);
    x->p_last = x->past + (int)c.group.div(x->row0 + x->rows - 1);
    const int keys = max(0, min(min(seq.ctx, c.capacity), x->p_last + 1));
    const int start = c.window ? (max(0, x->p_first - c.window + 1) & -c.step) : 0;
    x->k_lo = (int)min((int64_t)keys, start + ((int64_t)x->u0 << c.unit_log2));
    x->k_hi = (int)min((int64_t)keys, start + ((int64_t)x->u1 << c.unit_log2));
}

// Items taken whole, a workgroup each, which must not walk through many sequences
// (a batch's time would grow with its square).  The places of a kv head:
//   up to 64 sequences: their items one after the other (a load and a scan);
//   decode steps of more: ceil(group / rows) of each token, so those of sequence b
//     begin at query_start[b] ceil(group / rows);
//   others: a(b) = floor(query_start[b] group / rows) and on, a(b + 1) - a(b) items
//     of sequence b, which has one more at most (floor(A + B) - floor(A) is B rounded
//     down or up); behind all of those one place for each sequence's last item, at
//     min(query_start[b], b), which grows by 1 over a sequence with new tokens.
// The sequence of a place is the last that begins at it or in front, found as in
// last_low.  Empty places are behind the items, or (the last items of sequences) few
// among them: in their midst they would hold up workgroups with work (40 x 2 tokens
// of 1500 keys, 8 heads a kv head: 15.6 us, with an empty place behind each item 23.7).
// item_bound() counts them.
struct Places {
    // The kernel's loop over items is left after the first one and holds nothing for
    // others: no scalar registers are spilled for them (50 to 110 are for ranges).
    static constexpr bool once = true;
    Seq seq;

    // Picks the sequence of a place; false if the place is empty.
    __device__ __forceinline__ bool find(const Cut& c, const BatchArg& batch, uint32_t place, uint32_t* item) {
        const uint32_t x = c.kv_heads.div(place);
        uint32_t up;  // item of the kv head
        if (batch.seqs <= 64) {
            const int lane = threadIdx.x & 63;
            Seq s = {};
            if (lane < batch.seqs) read_sequence(c, batch, lane, &s);
            cut_sequence(c, &s);
            uint32_t sum = s.tiles;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t t = (uint32_t)__shfl_up((int)sum, o);
                if (lane >= o) sum += t;
            }
            const uint64_t past = __ballot(sum > x);
            if (!past) return false;
            const int l = __builtin_ctzll(past);
            seq.b = l;
            seq.row0 = __builtin_amdgcn_readlane(s.row0, l);
            seq.n = __builtin_amdgcn_readlane(s.n, l);
            seq.ctx = __builtin_amdgcn_readlane(s.ctx, l);
            cut_sequence(c, &seq);
            up = x - (uint32_t)__builtin_amdgcn_readlane((int)(sum - s.tiles), l);
        } else {
            auto start_of = [&](int b) { return (int64_t)max(batch.query_start[b], 0); };
            auto full = [&](int b) { return start_of(b) * c.group.d >> c.rows_log2; };
            const int64_t fulls = c.per_token ? 0 : full(batch.seqs);
            int b;
            if (c.per_token) {
                b = last_low(batch.seqs, [&](int j) { return start_of(j) * c.per_token <= x; });
                up = x - (uint32_t)(start_of(max(b, 0)) * c.per_token);
            } else if (x < fulls) {
                b = last_low(batch.seqs, [&](int j) { return full(j) <= x; });
                up = x - (uint32_t)full(max(b, 0));
            } else {
                b = last_low(batch.seqs, [&](int j) { return min(start_of(j), (int64_t)j) <= x - fulls; });
                up = (uint32_t)(full(max(b, 0) + 1) - full(max(b, 0)));
                if (min(start_of(max(b, 0)), (int64_t)max(b, 0)) != x - fulls) return false;
            }
            if (b < 0) return false;
            read_sequence(c, batch, b, &seq);
            cut_sequence(c, &seq);
        }
        *item = up * c.kv_heads.d + (place - x * c.kv_heads.d);
        return up < (uint32_t)seq.tiles;
    }
    // This workgroup's item, the only one.
    __device__ __forceinline__ bool start(const Cut& c, const BatchArg& batch, Item* x) {
        uint32_t item;
        if (!find(c, batch, c.place + blockIdx.x, &item)) return false;
        x->u0 = 0;
        x->u1 = seq.units;
        place_item(c, seq, item, x);
        place_keys(c, seq, x);
        return true;
    }
    __device__ __forceinline__ bool next(const Cut&, const BatchArg&, Item*) { return true; }
    __device__ __forceinline__ bool whole(const Item&) const { return true; }
};

// Ranges of units, as whole waves see them: each lane holds the lengths of one of
// 64 sequences (read once where there are no more), a wave's scan finds the
// sequence of a unit.  A workgroup walks through the sequences twice, but there
// are never more workgroups than the machine holds.
struct Work {
    static constexpr bool once = false;
    uint32_t total;  // units of all sequences
    uint32_t begin;  // first unit of seq
    Seq seq;
    uint32_t lo, hi;  // the units left of this workgroup's range

    int base;               // sequence of lane 0
    int l_row0, l_n, l_ctx; // this lane's sequence
    uint32_t l_units, l_sum; // its units, and those of the lanes up to it

    __device__ __forceinline__ void load(const Cut& c, const BatchArg& batch, int b0) {
        const int lane = threadIdx.x & 63;
        base = b0;
        Seq s = {};
        if (b0 + lane < batch.seqs) read_sequence(c, batch, b0 + lane, &s);
        cut_sequence(c, &s);
        l_row0 = s.row0;
        l_n = s.n;
        l_ctx = s.ctx;
        l_units = l_sum = c.kv_heads.d * s.tiles * s.units;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t t = (uint32_t)__shfl_up((int)l_sum, o);
            if (lane >= o) l_sum += t;
        }
    }
    __device__ __forceinline__ void pick(const Cut& c, const BatchArg& batch, int b) {
        if (b - base >= 64) load(c, batch, b);
        seq.b = b;
        seq.row0 = __builtin_amdgcn_readlane(l_row0, b - base);
        seq.n = __builtin_amdgcn_readlane(l_n, b - base);
        seq.ctx = __builtin_amdgcn_readlane(l_ctx, b - base);
        cut_sequence(c, &seq);
    }
    __device__ __forceinline__ void sum(const Cut& c, const BatchArg& batch) {
        total = 0;
        for (int b0 = 0; b0 < batch.seqs; b0 += 64) {
            load(c, batch, b0);
            total += (uint32_t)__builtin_amdgcn_readlane((int)l_sum, 63);
        }
    }
    // Picks the sequence that holds a unit (below total).
    __device__ __forceinline__ bool find(const Cut& c, const BatchArg& batch, uint32_t unit) {
        begin = 0;
        for (int b0 = 0; b0 < batch.seqs; b0 += 64) {
            if (base != b0) load(c, batch, b0);
            const uint64_t past = __ballot(begin + l_sum > unit);
            if (past) {
                const int l = __builtin_ctzll(past);
                begin += (uint32_t)__builtin_amdgcn_readlane((int)(l_sum - l_units), l);
                pick(c, batch, b0 + l);
                return true;
            }
            begin += (uint32_t)__builtin_amdgcn_readlane((int)l_sum, 63);
        }
        return false;
    }

    // This workgroup's range; next() goes through its items.
    __device__ __forceinline__ bool start(const Cut& c, const BatchArg& batch, Item*) {
        sum(c, batch);
        const uint32_t grid = min((uint32_t)gridDim.x, total);  // no range is empty
        if (blockIdx.x >= grid) return false;
        lo = range_begin(total, blockIdx.x, grid);
        hi = range_begin(total, blockIdx.x + 1, grid);
        return find(c, batch, lo);
    }
    __device__ __forceinline__ bool next(const Cut& c, const BatchArg& batch, Item* x) {
        if (lo >= hi) return false;
        while (lo - begin >= c.kv_heads.d * seq.tiles * seq.units) {
            begin += c.kv_heads.d * seq.tiles * seq.units;
            if (seq.b + 1 >= batch.seqs) return false;
            pick(c, batch, seq.b + 1);
        }
        const uint32_t item = seq.units == 1 ? lo - begin : (lo - begin) / (uint32_t)seq.units;
        x->u0 = (int)((lo - begin) - item * seq.units);
        x->u1 = (int)min((uint32_t)seq.units, x->u0 + (hi - lo));
        lo += x->u1 - x->u0;
        place_item(c, seq, item, x);
        place_keys(c, seq, x);
        return true;
    }
    __device__ __forceinline__ bool whole(const Item& x) const { return x.u0 == 0 && x.u1 == seq.units; }
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

// Bits [from, to) of 64, clamped to them.
__device__ __forceinline__ uint64_t bits_between(int from, int to) {
    const uint64_t below_to = to <= 0 ? 0 : to >= 64 ? ~uint64_t(0) : (uint64_t(1) << to) - 1;
    const uint64_t below_from = from <= 0 ? 0 : from >= 64 ? ~uint64_t(0) : (uint64_t(1) << from) - 1;
    return below_to & ~below_from;
}
// Bit i as 0 or ~0, and s where that is ~0, else -infinity: two vector
// operations and no lane masks (dozens of which would spill scalar registers).
__device__ __forceinline__ uint32_t bit_mask(uint32_t bits, int i) { return (uint32_t)__builtin_amdgcn_sbfe((int)bits, i, 1); }
__device__ __forceinline__ float keep_seen(float s, uint32_t mask) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, s) & mask) | (0xFF800000u & ~mask));
}

// 1 / sum of a row's weights, 0 for a row that sees no key (NaN stays NaN).
__device__ __forceinline__ float row_scale(float sum) { return sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f; }
// The natural log of 2^top * sum.
__device__ __forceinline__ float row_lse(float top, float sum) {
    return sum > 0.0f ? (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f : (sum != sum ? sum : kNone);
}

// l + both halves of p.
template <typename T>
__device__ __forceinline__ float add_pair(uint32_t p, float l) {
    if constexpr (std::is_same<T, F16>::value) {
        const h2 one = {(_Float16)1.0f, (_Float16)1.0f};
        return __builtin_amdgcn_fdot2(as_h2(p), one, l, false);
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        const b2 one = {(__bf16)1.0f, (__bf16)1.0f};
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, p), one, l, false);
    }
}

// Direct-to-LDS load from a wave's address and a lane's offset: lane i's 16
// bytes land at lds + 16 i.  Issued through asm so
// that the compiler does not wait for a tile in flight before it reads the
// other one; the kernel waits itself (vmcnt) before the tile's barrier.
__device__ __forceinline__ void load_to_lds(const char* src, uint32_t offset, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(src), "{m0}"(lds) : "memory");
}
// The same for lines that nobody reads again.
__device__ __forceinline__ void load_to_lds_once(const char* src, uint32_t offset, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(offset), "s"(src), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Two transposing reads (ds_read_b64_tr_b16): in each, 16 lanes give the places of
// 4 rows x 16 elements (lane i: 8 bytes, elements 4 (i % 4) .. of row i / 4), and
// lane i gets element i of the 4 rows.
__device__ __forceinline__ u4 read_transposed(const char* first, const char* second) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 l_s4;
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    const u2 x = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((l_s4*)first));
    const u2 y = __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((l_s4*)second));
    return u4{x.x, x.y, y.x, y.y};
}

// A head's row in LDS, as direct loads fill it: 1024 bytes a wave's load.
template <int D>
struct LdsRow {
    static constexpr int row = D <= 64 ? 128 : D <= 128 ? 256 : 512;  // bytes
    static constexpr int chunks = row / 16;                           // of 16 bytes
    static constexpr int per_load = 1024 / row;                       // rows of a load
    // XOR of a row's chunks for K, whose reads take one chunk of 16 rows: it
    // spreads those over all 64 banks.
    static __device__ __forceinline__ int swz_k(int r) { return chunks == 8 ? (r >> 1) & 7 : r & 15; }
};

}  // namespace q4

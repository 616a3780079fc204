// Arguments and launchers of the rotary, cache-append and attention kernels
// (internal to the library; the C ABI layer has validated everything here).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace q4 {

// Heads of a token list (strides in elements).
struct HeadsArg {
    char* data;
    int64_t token_stride, head_stride;
};

// Exact x / d for 0 <= x < 2^31 as one 64-bit product: with 2^(s-1) < d <= 2^s
// and mul = ceil(2^(31+s) / d), mul * d exceeds 2^(31+s) by less than d <= 2^s,
// so x * mul / 2^(31+s) exceeds x / d by less than x / 2^31 / d < 1 / d.
struct FastDiv {
    uint32_t d, mul;
    int shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t divisor) : d(divisor), mul(0), shift(31) {
        while ((uint64_t(1) << (shift - 31)) < divisor) ++shift;
        mul = (uint32_t)(((uint64_t(1) << shift) + divisor - 1) / divisor);
    }
#ifdef __HIPCC__
    __host__ __device__ __forceinline__ uint32_t div(uint32_t x) const { return (uint32_t)(((uint64_t)x * mul) >> shift); }
#endif
};

struct CacheArg {
    char* k;
    char* v;
    int64_t k_page, k_head, k_slot, v_page, v_head, v_slot;  // strides, elements
    uint32_t pages;
    FastDiv page_size;
    int kv_heads, head_dim;
};

struct BatchArg {
    const int32_t* table;
    int64_t table_stride;
    int table_pages, seqs;
    const int32_t* query_start;
    const int32_t* context_len;
};

// One launch of the rotary kernel: `nrot` token lists whose heads turn (each
// into a token list of its own, or into the cache's keys), and the values that
// are copied into the cache.  Types are Q4_TYPE_*.
struct RopeArgs {
    HeadsArg in[3];     // q (or x), k, v
    HeadsArg out;       // of in[0]
    int heads[3];       // heads of each list, 0: not there
    int paged;          // k and v go to the cache, positions may come from it
    CacheArg cache;
    BatchArg batch;
    const int32_t* positions;  // may be null when paged
    const double* inv_freq;
    int64_t tokens;
    int head_dim, rot_dim;
    float mscale;
};
hipError_t launch_rope(const RopeArgs& a, int in_type, int out_type, int layout, hipStream_t s);

// The same with a norm of each turned head first.
struct NormRopeArgs {
    RopeArgs rope;
    const char* gain[2];  // of the queries (or x), of the keys; null: ones
    int gain_type;
    float eps;
};
hipError_t launch_norm_rope(const NormRopeArgs& a, int in_type, int out_type, int layout, hipStream_t s);

// Whether every head can be read and written in 16-byte pieces of 8 elements that
// hold whole pairs, or whole runs of them (half layout).
inline bool rope_vectors(const RopeArgs& a, int in_bytes, int out_bytes, bool half) {
    auto heads_aligned = [](const HeadsArg& h, int bytes) {
        return ((uintptr_t)h.data & 15) == 0 && h.token_stride * bytes % 16 == 0 && h.head_stride * bytes % 16 == 0;
    };
    bool vec = a.head_dim % 8 == 0 && a.rot_dim % (half ? 16 : 8) == 0;
    for (int i = 0; i < 3; ++i)
        if (a.heads[i]) vec = vec && heads_aligned(a.in[i], in_bytes);
    if (a.heads[0]) vec = vec && heads_aligned(a.out, out_bytes);
    if (a.paged) {
        const CacheArg& c = a.cache;
        vec = vec && (((uintptr_t)c.k | (uintptr_t)c.v) & 15) == 0;
        vec = vec && (c.k_page | c.k_head | c.k_slot | c.v_page | c.v_head | c.v_slot) % 8 == 0;
    }
    return vec;
}

struct AttnArgs {
    HeadsArg q, out;
    float* lse;
    CacheArg cache;
    BatchArg batch;
    int64_t tokens;
    int q_heads, group;     // group: query heads of a kv head
    float scale_log2;       // scale * log2(e)
    int window;             // 0: none
    void* workspace;
};
// The same where each new token sees those of its sequence that its mask names.
struct TreeArgs : AttnArgs {
    const uint64_t* mask;  // [tokens][mask_words]
    int mask_words;
};
// How a call is cut: a rule on sizes alone, the same for the workspace's size
// and the launch.
struct AttnShape {
    int rows;      // query rows (token, head of the group) of one item: 16, 32 (k_attn), 64, 128, of trees 256 (k_attn_tile)
    int most_rows; // rows that an item has, as far as the caller knows
    int unit;      // keys of one unit of work
    int step;      // keys a kernel takes at a time
    int grid;      // workgroups of ranges of units
    int places;    // workgroups of items that are taken whole, 0: ranges of units
    int per_token; // places of a token and kv head, 0: by rows
    bool few;      // far fewer items than workgroups
    size_t bytes;  // workspace, 0 where every item is taken whole
};
bool attn_head_dim_ok(int head_dim);
AttnShape attn_shape(const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int window, int max_query, int max_context, bool tree = false);
size_t attn_most_bytes(int head_dim, int64_t rows);  // that any call with up to so many rows of a kv head takes
hipError_t launch_attention_tree(const TreeArgs& a, const AttnShape& shape, int type, hipStream_t s);
hipError_t launch_attention(const AttnArgs& a, const AttnShape& shape, int type, hipStream_t s);

}  // namespace q4

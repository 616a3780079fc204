// Device-side building blocks shared by the rotary, cache-append and attention
// kernels: element types, wave-wide sums, the places of tokens in a paged cache.
#pragma once

#include "kv_launch.h"
#include "q4_device.h"

namespace q4 {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));

// Element types: storage and conversion (to nearest, ties to even).
struct F16 {
    typedef _Float16 elem;
    static constexpr int bytes = 2;
};
struct BF16 {
    typedef __bf16 elem;
    static constexpr int bytes = 2;
};
struct F32 {
    typedef float elem;
    static constexpr int bytes = 4;
};

template <typename T, int V>
struct Vec {
    typedef typename T::elem type __attribute__((ext_vector_type(V)));
};

// V consecutive elements as floats; the vector forms read 16 bytes at a time.
template <typename T, int V>
__device__ __forceinline__ void load_elems(const char* p, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = (float)*reinterpret_cast<const typename T::elem*>(p);
    } else {
        const auto v = *reinterpret_cast<const typename Vec<T, V>::type*>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (float)v[i];
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_elems(char* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        *reinterpret_cast<typename T::elem*>(p) = (typename T::elem)x[0];
    } else {
        typename Vec<T, V>::type v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (typename T::elem)x[i];
        *reinterpret_cast<typename Vec<T, V>::type*>(p) = v;
    }
}

// Cosine and sine of position * inv_freq, times mscale: the angle as turns in
// binary64, reduced to [-1/2, 1/2] there, and what its rounding to binary32 leaves
// out added to first order.
__device__ __forceinline__ f2 turn_of(int position, double inv_freq, float mscale) {
    double turns = (double)position * inv_freq * 0.15915494309189533577;  // / (2 pi)
    turns -= __builtin_rint(turns);
    const float near = (float)turns;
    const float rest = 6.2831853071795864769f * (float)(turns - near);  // below 2^-22
    float s, c;
    sincospif(2.0f * near, &s, &c);
    return f2{(c - rest * s) * mscale, (s + rest * c) * mscale};
}

// The last j in [0, n) for which low(j) holds, where it holds for the first ones and
// not for the others; -1 if for none.  Called by whole waves with n uniform: 64
// places a step, counted with a ballot, so 64^k sequences take k loads one after
// the other (a walk through all of them would make a batch's time grow with its
// square, as every token and every item looks for its own).
template <typename F>
__device__ __forceinline__ int last_low(int n, F low) {
    const int lane = (int)(threadIdx.x & 63);
    int base = 0;
    for (;;) {
        const int step = (n + 63) >> 6;
        const int at = lane * step;
        const int count = __popcll(__ballot(at < n && low(base + at)));
        if (step <= 1 || !count) return base + count - 1;
        base += (count - 1) * step;
        n = min(step, n - (count - 1) * step);
    }
}

// The sequence whose new tokens hold row t: the last b with query_start[b] <= t
// (sequences without new tokens share their start with the next one), -1 for a
// row before the first or behind the last.  Called by whole waves with t uniform.
__device__ __forceinline__ int sequence_of(const BatchArg& b, int64_t t) {
    if (t >= b.query_start[b.seqs]) return -1;
    return last_low(b.seqs, [&](int j) { return b.query_start[j] <= t; });
}

// Page that holds position p of the sequence with block-table row `row`, or -1
// if the position has no place.
__device__ __forceinline__ int page_of(const CacheArg& c, const BatchArg& b, const int32_t* row, int p) {
    const uint32_t column = c.page_size.div((uint32_t)p);
    if (p < 0 || column >= (uint32_t)b.table_pages) return -1;
    const int page = row[column];
    return (uint32_t)page < c.pages ? page : -1;
}

}  // namespace q4

// Norms of heads with the rotation in the same pass, alone and on the way into a
// paged key/value cache (gfx950).
//
// For each head x of a token:  y = x g / sqrt(mean(x^2) + eps), then pairs of y turn by
// the token's angle as in rope.hip.  Everything from the read of x to the one rounding
// of the result is binary32 (the angle binary64): a norm that rounds y to the model's
// type first, as two separate passes would, loses half a step more.
//
// A group of L lanes (8 for heads of 128) holds a head in registers, 16 bytes of a
// 16-bit head a load; the sum of squares is joined by log2 L lane exchanges, and each
// lane turns the pairs it holds, so a head is read once and written once.  Angles are
// computed once a token and the gains read once a workgroup, into LDS; a workgroup has
// four tokens, whose heads are requested together.  Values (kv append) are copied by
// the same groups.
//
// Bound by memory for prompts and by latency for single tokens, as the rotation alone: a
// token of 32/8 heads of 128 from binary32 into an f16 cache 4.4 us (an empty launch 3.8),
// 5 ragged prompts of 6709 tokens, 32/8 heads, bf16, 34.4 us (165 MB read and written, 4.8
// TB/s; a large copy reaches 4.7).  The heads of four tokens are held as they were read,
// 16-bit ones packed, and one token's results are made at a time: held as binary32, with
// all tokens' results under way, they took twice the registers (41.5 us).
#include "kv_device.h"
#include "q4gemv.h"

#include <algorithm>

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;      // of a workgroup: one a wave in the setup
constexpr int kMaxPairs = 512;  // head_dim <= 1024

struct NormUnits {
    int rotating, units;       // units of a normed head that hold pairs, and all
    int heads, items;          // normed heads; with the pieces of values, L units each
    int value_units;           // units of a token's values
    FastDiv per_value;         // units of a value head
    int lanes_log2;            // L
    float inv_dim;
};

// V elements as they lie in memory.
template <typename T, int V>
struct Piece {
    typedef typename Vec<T, V>::type raw;
    raw v;
    __device__ __forceinline__ void clear() { v = raw(0); }
    __device__ __forceinline__ void load(const char* p) { v = *reinterpret_cast<const raw*>(p); }
    __device__ __forceinline__ float at(int i) const { return (float)v[i]; }
};
template <typename T>
struct Piece<T, 1> {
    typename T::elem v;
    __device__ __forceinline__ void clear() { v = (typename T::elem)0.0f; }
    __device__ __forceinline__ void load(const char* p) { v = *reinterpret_cast<const typename T::elem*>(p); }
    __device__ __forceinline__ float at(int) const { return (float)v; }
};
template <typename T, int V, int W>
__device__ __forceinline__ void store_pair(char* p, const float (&x)[W]) {
    if constexpr (V > 1) {
        store_elems<T, W>(p, x);
    } else {
        reinterpret_cast<typename T::elem*>(p)[0] = (typename T::elem)x[0];
        reinterpret_cast<typename T::elem*>(p)[1] = (typename T::elem)x[1];
    }
}

// Units as in k_rope: half layout: V elements from the first half and V from the second
// (or V that do not turn); interleaved: W consecutive ones.  NU units a lane.
template <typename IN, typename OUT, bool HALF, int V, int NU>
__global__ void __launch_bounds__(kThreads) k_norm_rope(const NormRopeArgs a, const NormUnits n) {
    constexpr int W = HALF ? V : (V < 2 ? 2 : V);
    constexpr int NP = HALF || V == 1 ? 2 : 1;  // pieces of a unit
    __shared__ f2 turn[kTokens][kMaxPairs];
    __shared__ float gain[2][2 * kMaxPairs];
    __shared__ int64_t place_k[kTokens], place_v[kTokens];
    __shared__ int state[kTokens];  // bit 0: the row is a token, bit 1: it has a place in the cache
    const RopeArgs& r = a.rope;
    const int64_t t0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * kTokens;
    {
        const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
        const int64_t t = t0 + w;
        int st = 0, p = 0;
        if (t < r.tokens) {
            st = 1;
            if (r.paged) {
                const int b = sequence_of(r.batch, t);
                st = b >= 0;
                if (b >= 0) {
                    p = r.batch.context_len[b] - r.batch.query_start[b + 1] + (int)t;
                    const int page = page_of(r.cache, r.batch, r.batch.table + b * r.batch.table_stride, p);
                    if (page >= 0) {
                        st = 3;
                        const int64_t slot = p - (int64_t)r.cache.page_size.div((uint32_t)p) * r.cache.page_size.d;
                        if (lane == 0) {
                            place_k[w] = page * r.cache.k_page + slot * r.cache.k_slot;
                            place_v[w] = page * r.cache.v_page + slot * r.cache.v_slot;
                        }
                    }
                }
            }
            if (r.positions) p = r.positions[t];
        }
        if (lane == 0) state[w] = st;
        if (st)
            for (int i = lane; i < r.rot_dim / 2; i += 64) turn[w][i] = turn_of(p, r.inv_freq[i], r.mscale);
        for (int i = threadIdx.x; i < 2 * r.head_dim; i += kThreads) {
            const int which = i >= r.head_dim, e = i - which * r.head_dim;
            const char* g = a.gain[which];
            float v = 1.0f;
            if (g) {
                if (a.gain_type == Q4_TYPE_F32)
                    v = reinterpret_cast<const float*>(g)[e];
                else if (a.gain_type == Q4_TYPE_F16)
                    v = (float)reinterpret_cast<const _Float16*>(g)[e];
                else
                    v = (float)reinterpret_cast<const __bf16*>(g)[e];
            }
            gain[which][e] = v;
        }
    }
    __syncthreads();
    const int half = r.rot_dim / 2;
    const int lane = threadIdx.x & ((1 << n.lanes_log2) - 1);
    const int groups = kThreads >> n.lanes_log2;
    // (whole waves stay in the loop: the lanes of a group exchange sums)
    for (int at = blockIdx.y * groups; at < n.items; at += gridDim.y * groups) {
        const int item = at + (int)(threadIdx.x >> n.lanes_log2);
        if (item >= n.heads) {
            if (item >= n.items) continue;
            // values: copied
#pragma unroll 1
            for (int j = 0; j < NU; ++j) {
                const int u = (((item - n.heads) * NU + j) << n.lanes_log2) + lane;
                if (u >= n.value_units) break;
                const int h = (int)n.per_value.div((uint32_t)u), e = (u - h * (int)n.per_value.d) * V;
                float v[kTokens][V];
#pragma unroll
                for (int k = 0; k < kTokens; ++k) {
                    const int64_t t = t0 + k < r.tokens ? t0 + k : r.tokens - 1;
                    load_elems<IN, V>(r.in[2].data + (t * r.in[2].token_stride + h * r.in[2].head_stride + e) * IN::bytes, v[k]);
                }
#pragma unroll
                for (int k = 0; k < kTokens; ++k)
                    if (state[k] & 2) store_elems<OUT, V>(r.cache.v + (place_v[k] + h * r.cache.v_head + e) * OUT::bytes, v[k]);
            }
            continue;
        }
        const int list = item >= r.heads[0], h = item - (list ? r.heads[0] : 0);
        const HeadsArg in = list ? r.in[1] : r.in[0];
        // All tokens' elements are read before any is written: out may be x itself.  They are
        // held as they are read (16-bit ones packed) and converted twice.
        Piece<IN, V> x[kTokens][NU][NP];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int64_t t = t0 + k < r.tokens ? t0 + k : r.tokens - 1;
            const char* src = in.data + (t * in.token_stride + h * in.head_stride) * IN::bytes;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int i = lane + (j << n.lanes_log2);
#pragma unroll
                for (int e = 0; e < NP; ++e) x[k][j][e].clear();
                if (i >= n.units) continue;
                const bool turns = i < n.rotating;
                const int e0 = turns ? i * (HALF ? V : W) : r.rot_dim + (i - n.rotating) * V;
                x[k][j][0].load(src + e0 * IN::bytes);
                if (NP == 2 && turns) x[k][j][NP - 1].load(src + (e0 + (HALF ? half : 1)) * IN::bytes);
            }
        }
        float scale[kTokens];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < NU; ++j)
#pragma unroll
                for (int e = 0; e < NP * V; ++e) {
                    const float v = x[k][j][e / V].at(e % V);
                    sum = __builtin_fmaf(v, v, sum);
                }
            scale[k] = sum;
        }
        for (int o = 1; o < 1 << n.lanes_log2; o <<= 1)
#pragma unroll
            for (int k = 0; k < kTokens; ++k) scale[k] += __shfl_xor(scale[k], o);
#pragma unroll
        for (int k = 0; k < kTokens; ++k) scale[k] = 1.0f / __builtin_sqrtf(scale[k] * n.inv_dim + a.eps);
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            __builtin_amdgcn_sched_barrier(0);  // registers: one token's results at a time
            const int st = state[k];
            if (!(list == 0 ? st & 1 : st & 2)) continue;
            char* dst = list == 0 ? r.out.data + ((t0 + k) * r.out.token_stride + h * r.out.head_stride) * OUT::bytes
                                  : r.cache.k + (place_k[k] + h * r.cache.k_head) * OUT::bytes;
#pragma unroll
            for (int j = 0; j < NU; ++j) {
                const int i = lane + (j << n.lanes_log2);
                if (i >= n.units) continue;
                const bool turns = i < n.rotating;
                const int e0 = turns ? i * (HALF ? V : W) : r.rot_dim + (i - n.rotating) * V;
                const float* g = &gain[list][e0];
                const Piece<IN, V>*y = x[k][j];
                if (turns) {
                    const f2* cs = &turn[k][HALF ? e0 : e0 / 2];
                    if (HALF) {
                        float lo[V], hi[V];
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float p = y[0].at(e) * scale[k] * g[e], q = y[NP - 1].at(e) * scale[k] * g[half + e];
                            lo[e] = p * cs[e].x - q * cs[e].y;
                            hi[e] = p * cs[e].y + q * cs[e].x;
                        }
                        store_elems<OUT, V>(dst + e0 * OUT::bytes, lo);
                        store_elems<OUT, V>(dst + (e0 + half) * OUT::bytes, hi);
                    } else {
                        float o[W];
#pragma unroll
                        for (int e = 0; e < W / 2; ++e) {
                            const float p = (V > 1 ? y[0].at(V > 1 ? 2 * e : 0) : y[0].at(0)) * scale[k] * g[2 * e];
                            const float q = (V > 1 ? y[0].at(V > 1 ? 2 * e + 1 : 0) : y[NP - 1].at(0)) * scale[k] * g[2 * e + 1];
                            o[2 * e] = p * cs[e].x - q * cs[e].y;
                            o[2 * e + 1] = p * cs[e].y + q * cs[e].x;
                        }
                        store_pair<OUT, V>(dst + e0 * OUT::bytes, o);
                    }
                } else {
                    float o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = y[0].at(e) * scale[k] * g[e];
                    store_elems<OUT, V>(dst + e0 * OUT::bytes, o);
                }
            }
        }
    }
}

template <typename IN, typename OUT, bool HALF, int V, int NU>
hipError_t launch_units(const NormRopeArgs& a, NormUnits n, hipStream_t s) {
    const RopeArgs& r = a.rope;
    const int groups = kThreads >> n.lanes_log2;
    n.items = n.heads + (n.value_units + (NU << n.lanes_log2) - 1) / (NU << n.lanes_log2);
    const int64_t bx = (r.tokens + kTokens - 1) / kTokens;
    // Few tokens: a token's heads over several workgroups.
    const int64_t want = (1024 + bx - 1) / bx;
    const int by = (int)std::max<int64_t>(1, std::min<int64_t>(want, (n.items + groups - 1) / groups));
    // a launch has fewer than 2^32 threads along each axis
    const unsigned gx = (unsigned)std::min<int64_t>(bx, 1 << 22), gz = (unsigned)((bx + gx - 1) / gx);
    hipLaunchKernelGGL((k_norm_rope<IN, OUT, HALF, V, NU>), dim3(gx, (unsigned)by, gz), dim3(kThreads), 0, s, a, n);
    return hipGetLastError();
}

template <typename IN, typename OUT, bool HALF, int V>
hipError_t launch(const NormRopeArgs& a, hipStream_t s) {
    constexpr int W = HALF ? V : (V < 2 ? 2 : V);
    const RopeArgs& r = a.rope;
    NormUnits n = {};
    n.rotating = HALF ? r.rot_dim / 2 / V : r.rot_dim / W;
    n.units = n.rotating + (r.head_dim - r.rot_dim) / V;
    n.heads = r.heads[0] + r.heads[1];
    n.value_units = r.heads[2] * (r.head_dim / V);
    n.per_value = FastDiv((uint32_t)(r.head_dim / V));
    n.inv_dim = 1.0f / (float)r.head_dim;
    // as few lanes as hold a head at a unit each, a wave at most
    while (n.lanes_log2 < 6 && 1 << n.lanes_log2 < n.units) ++n.lanes_log2;
    const int each = (n.units + (1 << n.lanes_log2) - 1) >> n.lanes_log2;
    if constexpr (V == 8)
        return each == 1 ? launch_units<IN, OUT, HALF, V, 1>(a, n, s) : launch_units<IN, OUT, HALF, V, 2>(a, n, s);
    else
        return each <= 4 ? launch_units<IN, OUT, HALF, V, 4>(a, n, s) : launch_units<IN, OUT, HALF, V, 16>(a, n, s);
}

template <typename IN, typename OUT>
hipError_t launch_types(const NormRopeArgs& a, int layout, hipStream_t s) {
    const bool half = layout == Q4_ROPE_HALF, vec = rope_vectors(a.rope, IN::bytes, OUT::bytes, half);
    if (half) return vec ? launch<IN, OUT, true, 8>(a, s) : launch<IN, OUT, true, 1>(a, s);
    return vec ? launch<IN, OUT, false, 8>(a, s) : launch<IN, OUT, false, 1>(a, s);
}

template <typename IN>
hipError_t launch_out(const NormRopeArgs& a, int out_type, int layout, hipStream_t s) {
    if (out_type == Q4_TYPE_F16) return launch_types<IN, F16>(a, layout, s);
    if (out_type == Q4_TYPE_BF16) return launch_types<IN, BF16>(a, layout, s);
    return launch_types<IN, F32>(a, layout, s);
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, int in_type, int out_type, int layout, hipStream_t s) {
    if (in_type == Q4_TYPE_F16) return launch_out<F16>(a, out_type, layout, s);
    if (in_type == Q4_TYPE_BF16) return launch_out<BF16>(a, out_type, layout, s);
    return launch_out<F32>(a, out_type, layout, s);
}

}  // namespace q4

// Rotary positions, alone and on the way into a paged key/value cache (gfx950).
//
// Pair i of a head is turned by the angle positions[t] * inv_freq[i]:
//   (a, b) -> m (a cos - b sin, a sin + b cos).
// An angle of a far position keeps only its last bits modulo a turn, so it is
// formed in binary64 as a number of turns, reduced to [-1/2, 1/2] there, and
// only then taken to binary32 for the sine and cosine; what that leaves out, up to
// 2^-26 of a turn, turns them on to first order (binary32 outputs would see it: an
// rms error of 0.65 of 2^-24 of a pair's length instead of 0.49, which rounded
// sines and cosines alone give).  They are the same for every head of a token:
// each wave computes one token's into LDS, and the workgroup's threads then turn
// all heads of its tokens, 16 bytes of a 16-bit head per load and store.
//
// The work is one read and one write of the heads, so a prompt is bound by
// memory; a decode step's tokens are bound by latency (start, sequence search,
// block table, store), and then the units of a token are spread over several
// workgroups.
//
// Measured with 12 sets of tensors in turn, more than the last-level cache holds:
// 8191 tokens of 32 heads of 128, 64 of each rotated, in bf16 30.3 us (4.4 TB/s read
// and written; a plain copy of the same heads 27.1), rotated whole in binary32 55.4
// us (4.9 TB/s), 5 ragged prompts of 6,709 tokens together into a cache of 8 heads
// with 32 query heads 39.5 us (4.2 TB/s); with one set, from that cache in part,
// 23.1, 47.8 and 30.7 us.  One token 3.7 to 4.1 us, as long as an empty launch.
#include "kv_device.h"
#include "q4gemv.h"

#include <algorithm>

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;     // tokens of a workgroup: one a wave in the setup
constexpr int kMaxPairs = 512; // head_dim <= 1024

struct RopeUnits {
    FastDiv per_head, per_value;  // units of a turned head, of a copied head
    int rotating;                 // units of a head that hold pairs
    int units[3];                 // units of a token in each list
};

// Elements of one unit of work in half layout: V from the first half and V from
// the second (or V copied ones); interleaved: W = max(V, 2) consecutive ones.
template <typename IN, typename OUT, bool HALF, int V>
__global__ void __launch_bounds__(kThreads) k_rope(const RopeArgs a, const RopeUnits n) {
    constexpr int W = HALF ? V : (V < 2 ? 2 : V);
    constexpr int E = HALF ? 2 * V : W;
    __shared__ f2 turn[kTokens][kMaxPairs];
    __shared__ int64_t place_k[kTokens], place_v[kTokens];
    __shared__ int state[kTokens];  // bit 0: the row is a token, bit 1: it has a place in the cache
    const int64_t t0 = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * kTokens;
    {
        const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
        const int64_t t = t0 + w;
        int st = 0, p = 0;
        if (t < a.tokens) {
            st = 1;
            if (a.paged) {
                const int b = sequence_of(a.batch, t);
                st = b >= 0;
                if (b >= 0) {
                    p = a.batch.context_len[b] - a.batch.query_start[b + 1] + (int)t;
                    const int page = page_of(a.cache, a.batch, a.batch.table + b * a.batch.table_stride, p);
                    if (page >= 0) {
                        st = 3;
                        const int64_t slot = p - (int64_t)a.cache.page_size.div((uint32_t)p) * a.cache.page_size.d;
                        if (lane == 0) {
                            place_k[w] = page * a.cache.k_page + slot * a.cache.k_slot;
                            place_v[w] = page * a.cache.v_page + slot * a.cache.v_slot;
                        }
                    }
                }
            }
            if (a.positions) p = a.positions[t];
        }
        if (lane == 0) state[w] = st;
        if (st) {
            for (int i = lane; i < a.rot_dim / 2; i += 64) {
                turn[w][i] = turn_of(p, a.inv_freq[i], a.mscale);
            }
        }
    }
    __syncthreads();
    const int total = n.units[0] + n.units[1] + n.units[2];
    const int half = a.rot_dim / 2;
    for (int u = blockIdx.y * kThreads + threadIdx.x; u < total; u += gridDim.y * kThreads) {
        const int list = u < n.units[0] ? 0 : u < n.units[0] + n.units[1] ? 1 : 2;
        const int r = u - (list == 0 ? 0 : list == 1 ? n.units[0] : n.units[0] + n.units[1]);
        const FastDiv& per = list == 2 ? n.per_value : n.per_head;
        const int h = (int)per.div((uint32_t)r);
        const int i = r - h * (int)per.d;
        const bool turns = list != 2 && i < n.rotating;
        // first element, and (half layout) the distance to its partner
        const int e = turns ? i * (HALF ? V : W) : list == 2 ? i * V : a.rot_dim + (i - n.rotating) * V;
        const HeadsArg in = list == 0 ? a.in[0] : list == 1 ? a.in[1] : a.in[2];
        // all tokens' elements are read before any is written: out may be x itself
        float x[kTokens][E];
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int64_t t = t0 + k < a.tokens ? t0 + k : a.tokens - 1;
            const char* src = in.data + (t * in.token_stride + h * in.head_stride + e) * IN::bytes;
            if (!HALF && turns) {
                float v[W];
                load_elems<IN, W>(src, v);
#pragma unroll
                for (int j = 0; j < W; ++j) x[k][j] = v[j];
            } else {
                float v[V];
                load_elems<IN, V>(src, v);
#pragma unroll
                for (int j = 0; j < V; ++j) x[k][j] = v[j];
                if (HALF && turns) {
                    load_elems<IN, V>(src + half * IN::bytes, v);
#pragma unroll
                    for (int j = 0; j < V; ++j) x[k][(HALF ? V : 0) + j] = v[j];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kTokens; ++k) {
            const int st = state[k];
            if (!(list == 0 ? st & 1 : st & 2)) continue;
            char* dst;
            if (list == 0)
                dst = a.out.data + ((t0 + k) * a.out.token_stride + h * a.out.head_stride + e) * OUT::bytes;
            else if (list == 1)
                dst = a.cache.k + (place_k[k] + h * a.cache.k_head + e) * OUT::bytes;
            else
                dst = a.cache.v + (place_v[k] + h * a.cache.v_head + e) * OUT::bytes;
            if (turns) {
                const f2* cs = &turn[k][HALF ? e : e / 2];
                if (HALF) {
                    float lo[V], hi[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float p = x[k][j], q = x[k][(HALF ? V : 0) + j];
                        lo[j] = p * cs[j].x - q * cs[j].y;
                        hi[j] = p * cs[j].y + q * cs[j].x;
                    }
                    store_elems<OUT, V>(dst, lo);
                    store_elems<OUT, V>(dst + half * OUT::bytes, hi);
                } else {
                    float o[W];
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) {
                        const float p = x[k][2 * j], q = x[k][2 * j + (W > 1)];
                        o[2 * j] = p * cs[j].x - q * cs[j].y;
                        o[2 * j + (W > 1)] = p * cs[j].y + q * cs[j].x;
                    }
                    store_elems<OUT, W>(dst, o);
                }
            } else {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = x[k][j];
                store_elems<OUT, V>(dst, o);
            }
        }
    }
}

template <typename IN, typename OUT, bool HALF, int V>
hipError_t launch(const RopeArgs& a, hipStream_t s) {
    constexpr int W = HALF ? V : (V < 2 ? 2 : V);
    RopeUnits n;
    n.rotating = HALF ? a.rot_dim / 2 / V : a.rot_dim / W;
    const int per_head = n.rotating + (a.head_dim - a.rot_dim) / V;
    n.per_head = FastDiv((uint32_t)per_head);
    n.per_value = FastDiv((uint32_t)(a.head_dim / V));
    n.units[0] = a.heads[0] * per_head;
    n.units[1] = a.heads[1] * per_head;
    n.units[2] = a.heads[2] * (a.head_dim / V);
    const int total = n.units[0] + n.units[1] + n.units[2];
    const int64_t bx = (a.tokens + kTokens - 1) / kTokens;
    // Few tokens: a token's units over several workgroups, one unit a thread.
    const int64_t want = (1024 + bx - 1) / bx;
    const int by = (int)std::max<int64_t>(1, std::min<int64_t>(want, (total + kThreads - 1) / kThreads));
    // a launch has fewer than 2^32 threads along each axis
    const unsigned gx = (unsigned)std::min<int64_t>(bx, 1 << 22), gz = (unsigned)((bx + gx - 1) / gx);
    hipLaunchKernelGGL((k_rope<IN, OUT, HALF, V>), dim3(gx, (unsigned)by, gz), dim3(kThreads), 0, s, a, n);
    return hipGetLastError();
}

template <typename IN, typename OUT>
hipError_t launch_types(const RopeArgs& a, int layout, hipStream_t s) {
    const bool half = layout == Q4_ROPE_HALF, vec = rope_vectors(a, IN::bytes, OUT::bytes, half);
    if (half) return vec ? launch<IN, OUT, true, 8>(a, s) : launch<IN, OUT, true, 1>(a, s);
    return vec ? launch<IN, OUT, false, 8>(a, s) : launch<IN, OUT, false, 1>(a, s);
}

template <typename IN>
hipError_t launch_out(const RopeArgs& a, int out_type, int layout, hipStream_t s) {
    if (out_type == Q4_TYPE_F16) return launch_types<IN, F16>(a, layout, s);
    if (out_type == Q4_TYPE_BF16) return launch_types<IN, BF16>(a, layout, s);
    return launch_types<IN, F32>(a, layout, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int in_type, int out_type, int layout, hipStream_t s) {
    if (in_type == Q4_TYPE_F16) return launch_out<F16>(a, out_type, layout, s);
    if (in_type == Q4_TYPE_BF16) return launch_out<BF16>(a, out_type, layout, s);
    return launch_out<F32>(a, out_type, layout, s);
}

}  // namespace q4

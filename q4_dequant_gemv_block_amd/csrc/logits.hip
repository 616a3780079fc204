// Penalties, biases and grammars on rows of logits, and the greedy pick (gfx950).
//
// For row t and token v, with c the number of times v is among the answer's tokens and
// "seen" whether v is among the prompt's or the answer's:
//   x = seen ? (x > 0 ? x / repetition : x * repetition) : x
//   x = x - frequency c - (c > 0 ? presence : 0) + bias[v],  -infinity if not allowed,
// each step rounded to binary32 by itself, so that equal logits under equal rules stay
// equal and ties are decided by the index.  The pick is the lowest index among the
// largest; NaN and -infinity are never picked.
//
// A workgroup takes a slice of one row's vocabulary.  Its logits are requested first;
// while they are on their way the history is scanned once and the tokens of the slice
// counted in LDS (whole numbers: the order of the atomics does not matter; a bias
// keeps its largest place in the list, so the last of equal tokens counts).  Counting
// in the kernel keeps a sequence's state to its text: counts by vocabulary would be
// read and written with every step, four bytes for each logit.  The slices' keys
// (argmax_key) are joined by a second launch, a wave a row.
//
// Bound by memory in large batches (a slice of 8192 logits, the history from the L2),
// by latency and the two launches in small ones (slices of 1024, so that one row is
// read by 149 CUs).
#include "attn_device.h"
#include "step_launch.h"
#include "q4gemv.h"

#include <algorithm>

namespace q4 {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kPrompt = 0x80000000u;

// Four consecutive logits at any alignment of the type.
template <typename T>
struct Quad;
template <>
struct Quad<F32> {
    typedef float type __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Quad<F16> {
    typedef _Float16 type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Quad<BF16> {
    typedef __bf16 type __attribute__((ext_vector_type(4), aligned(2)));
};

__device__ __forceinline__ float none() { return -__builtin_inff(); }
__device__ __forceinline__ float not_a_number() { return __builtin_nanf(""); }
__device__ __forceinline__ int32_t token_of(uint64_t key) { return key ? (int32_t)(0xFFFFFFFFu - (uint32_t)key) : -1; }

// A product that no sum behind it takes in unrounded.
__device__ __forceinline__ float rounded(float v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The sequence of row t, -1 for a row in front of the first or behind the last.
__device__ __forceinline__ int sequence_of_rows(const LogitArgs& a, int64_t t) {
    if (t >= a.query_start[a.seqs]) return -1;
    return last_low(a.seqs, [&](int j) { return a.query_start[j] <= t; });
}

// NQ quads a thread: quad k of thread i holds the slice's logits 4 (256 k + i) .. .
// LISTS: there is a history, drafted tokens or biases.
template <typename T, int NQ, bool LISTS>
__global__ void __launch_bounds__(kThreads) k_logits(const LogitArgs a, int64_t total) {
    constexpr int kSlice = 4 * kThreads * NQ;
    extern __shared__ uint32_t lists[];  // counts [kSlice], then places of biases [kSlice]
    __shared__ uint64_t sh[kThreads / 64];
    uint32_t* count = lists;
    uint32_t* place = lists + kSlice;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int64_t t = u / a.slices;
        const int64_t lo = (u - t * a.slices) * kSlice;
        const int size = (int)min((int64_t)kSlice, a.vocab - lo);
        const char* row = a.logits + (t * a.row_stride + lo) * T::bytes;
        float x[NQ][4];
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int v = 4 * (kThreads * k + (int)threadIdx.x);
            if (v + 4 <= size) {
                const auto q = *reinterpret_cast<const typename Quad<T>::type*>(row + v * T::bytes);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k][e] = (float)q[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[k][e] = not_a_number();
                    if (v + e < size) x[k][e] = (float)*reinterpret_cast<const typename T::elem*>(row + (v + e) * T::bytes);
                }
            }
        }
        int64_t seq = t;
        int first = 0, n = 1;  // rows of the sequence
        if (a.query_start) {
            seq = sequence_of_rows(a, t);
            if (seq < 0) continue;  // the same for the whole workgroup
            first = a.query_start[seq];
            n = a.query_start[seq + 1] - first;
        } else {
            first = (int)t;
        }
        float repetition = 1.0f, presence = 0.0f, frequency = 0.0f;
        if (a.repetition) repetition = a.repetition[seq];
        if (a.presence) presence = a.presence[seq];
        if (a.frequency) frequency = a.frequency[seq];
        int bias0 = 0, bias1 = 0;
        if constexpr (LISTS) {
            if (a.bias_start) {
                bias0 = (int)min(max((int64_t)a.bias_start[seq], (int64_t)0), a.biases);
                bias1 = (int)min(max((int64_t)a.bias_start[seq + 1], (int64_t)bias0), a.biases);
            }
            const int words = a.bias_start ? 2 * kSlice : kSlice;
            for (int i = 4 * threadIdx.x; i < words; i += 4 * kThreads) *reinterpret_cast<u4*>(&lists[i]) = u4{0, 0, 0, 0};
            __syncthreads();
            auto note = [&](int token, bool answer) {
                const int64_t v = token - lo;
                if (v < 0 || v >= size) return;
                if (answer)
                    atomicAdd(&count[v], 1u);
                else
                    atomicOr(&count[v], kPrompt);
            };
            if (a.history) {
                const int len = min(a.history_len[seq], a.history_tokens), prompt = a.prompt_len ? a.prompt_len[seq] : 0;
                const int32_t* text = a.history + seq * a.history_stride;
                for (int i = threadIdx.x; i < len; i += 4 * kThreads) {
                    int token[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) token[e] = i + e * kThreads < len ? text[i + e * kThreads] : -1;
#pragma unroll
                    for (int e = 0; e < 4; ++e) note(token[e], i + e * kThreads >= prompt);
                }
            }
            if (a.draft) {
                const int own = (int)(t - first);
                const int most = a.mask ? min(n, 64 * a.mask_words) : own + 1;
                for (int j = threadIdx.x; j < most; j += kThreads)
                    if (first + (int64_t)j >= 0 && first + (int64_t)j < a.rows && (!a.mask || ((a.mask[t * a.mask_words + (j >> 6)] >> (j & 63)) & 1)))
                        note(a.draft[first + j], true);
            }
            for (int i = bias0 + threadIdx.x; i < bias1; i += kThreads) {
                const int64_t v = a.bias_tokens[i] - lo;
                if (v >= 0 && v < size) atomicMax(&place[v], (uint32_t)(i - bias0) + 1u);
            }
            __syncthreads();
        }
        const uint32_t* allowed = nullptr;
        if (a.allowed) {
            const int64_t r = a.allowed_row ? a.allowed_row[t] : t;
            if (r >= 0 && r < a.allowed_rows) allowed = a.allowed + r * a.allowed_stride + (lo >> 5);
        }
        float best = none();
        int at = 0;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int v = 4 * (kThreads * k + (int)threadIdx.x);
            if (v >= size) break;
            const uint32_t open = allowed ? allowed[v >> 5] >> (v & 31) : 15u;
            if constexpr (LISTS) {
                const u4 c4 = *reinterpret_cast<const u4*>(&count[v]);
                if (c4.x | c4.y | c4.z | c4.w) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t c = c4[e];
                        if (!c) continue;
                        const float answers = (float)(c & ~kPrompt);
                        float y = x[k][e];
                        if (a.repetition) y = rounded(y > 0.0f ? y / repetition : y * repetition);
                        y = y - rounded(frequency * answers);
                        if (c & ~kPrompt) y = y - presence;
                        x[k][e] = y;
                    }
                }
                if (bias1 > bias0) {
                    const u4 p4 = *reinterpret_cast<const u4*>(&place[v]);
                    if (p4.x | p4.y | p4.z | p4.w) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (p4[e]) x[k][e] = x[k][e] + a.bias_values[bias0 + p4[e] - 1];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = (open >> e) & 1 ? x[k][e] : none();
                x[k][e] = y;
                if (y > best && v + e < size) {
                    best = y;
                    at = v + e;
                }
            }
            if (a.out) {
                float* dst = a.out + t * a.out_stride + lo + v;
                if (v + 4 <= size) {
                    *reinterpret_cast<Quad<F32>::type*>(dst) = Quad<F32>::type{x[k][0], x[k][1], x[k][2], x[k][3]};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (v + e < size) dst[e] = x[k][e];
                }
            }
        }
        const uint64_t key = best > none() ? argmax_key(best, lo + at) : 0;
        const uint64_t top = block_max_u64(key, sh);
        if (threadIdx.x == 0) {
            if (a.slices == 1)
                a.tokens[t] = token_of(top);
            else
                a.keys[t * a.slices + (u - t * a.slices)] = top;
        }
        __syncthreads();  // lists and sh are read before the next slice's
    }
}

// tokens[t] from the keys of row t's slices, a wave a row.
__global__ void __launch_bounds__(kThreads) k_logits_pick(const LogitArgs a) {
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); t < a.rows; t += (int64_t)gridDim.x * (kThreads / 64)) {
        if (a.query_start && (t < a.query_start[0] || t >= a.query_start[a.seqs])) continue;
        uint64_t best = 0;
        for (int64_t s = lane; s < a.slices; s += 64) {
            const uint64_t v = a.keys[t * a.slices + s];
            best = v > best ? v : best;
        }
        best = wave_max_u64(best);
        if (lane == 0) a.tokens[t] = token_of(best);
    }
}

template <typename T, int NQ, bool LISTS>
hipError_t launch(const LogitArgs& a, hipStream_t s) {
    const int64_t total = a.rows * a.slices;
    const unsigned grid = (unsigned)std::min<int64_t>(total, 1 << 22);
    const size_t lds = LISTS ? (size_t)4 * kThreads * NQ * 4 * (a.bias_start ? 2 : 1) : 0;
    if constexpr (LISTS && NQ == 8) {  // 64 KiB and a little
        static LdsLimit limit;
        const hipError_t e = limit.raise(reinterpret_cast<const void*>(k_logits<T, NQ, LISTS>), lds + 1024);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_logits<T, NQ, LISTS>), dim3(grid), dim3(kThreads), lds, s, a, total);
    if (a.slices > 1) {
        const unsigned waves = kThreads / 64;
        hipLaunchKernelGGL(k_logits_pick, dim3((unsigned)std::min<int64_t>((a.rows + waves - 1) / waves, 1 << 20)), dim3(kThreads), 0, s, a);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t launch_type(const LogitArgs& a, hipStream_t s) {
    const bool lists = a.history || a.draft || a.bias_start;
    switch (logit_slice(a.rows, a.vocab)) {
        case 1024: return lists ? launch<T, 1, true>(a, s) : launch<T, 1, false>(a, s);
        case 2048: return lists ? launch<T, 2, true>(a, s) : launch<T, 2, false>(a, s);
        case 4096: return lists ? launch<T, 4, true>(a, s) : launch<T, 4, false>(a, s);
        default: return lists ? launch<T, 8, true>(a, s) : launch<T, 8, false>(a, s);
    }
}

}  // namespace

// As long a slice as leaves 4 workgroups a CU: each scans its row's history.
int64_t logit_slice(int64_t rows, int64_t vocab) {
    int64_t slice = 8192;
    while (slice > 1024 && rows * ((vocab + slice - 1) / slice) < 1024) slice /= 2;
    return slice;
}

hipError_t launch_logits(LogitArgs a, int type, hipStream_t s) {
    const int64_t slice = logit_slice(a.rows, a.vocab);
    a.slices = (a.vocab + slice - 1) / slice;
    if (type == Q4_TYPE_F16) return launch_type<F16>(a, s);
    if (type == Q4_TYPE_BF16) return launch_type<BF16>(a, s);
    return launch_type<F32>(a, s);
}

}  // namespace q4

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
// A workgroup takes a slice of one row's vocabulary.  Its logits are requested first,
// then the row's lists, all before any is waited for; the tokens of the slice are
// counted in LDS (whole numbers: the order of the atomics does not matter; then, in the
// same place, a bias keeps its largest place in the list, so the last of equal tokens
// counts).  Counting in the kernel keeps a sequence's state to its text: counts by
// vocabulary would be read and written with every step, four bytes for each logit.  The
// keys (argmax_key) of the slices' waves are joined by a second launch, a wave a row;
// joining in the first one would need counters that are zero before every call.
//
// Bound by memory in large batches: 192 rows of 151936 binary32 logits, each with up to
// 4096 tokens and 300 biases, read and written in 51 us of kernel time (4.6 TB/s; a
// copy of them takes 45, the bare pick with its copy 46).  Bound by latency in small
// ones: the sequence, its lengths, the lists and the counts follow each other, 4.9 us for
// one row, 13 for 37 rows of trees, and 2 to 4 for the second launch.  What made the
// difference (65 us before): lengths and penalties as scalar loads (as vector loads each
// waited for the logits), a quad's penalties without branches, and biases whose values
// are in the cells before they are added.  Rows one after the other in a workgroup, the
// next one's logits requested early, need registers that cost a third of the waves: 83 us.
#include "kv_device.h"
#include "step_launch.h"
#include "q4gemv.h"

#include <algorithm>

namespace q4 {

namespace {

constexpr int kThreads = 256;  // of the pick
constexpr uint32_t kPrompt = 0x80000000u;
constexpr uint32_t kNoBias = 0x80000000u;  // below any place; as a binary32 -0, which changes no sum
constexpr int kKeys = kLogitKeys;  // of a slice: its waves'

// Four consecutive logits at any alignment of the type.
template <typename E>
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

// The same for the whole workgroup, from a tensor that the call does not write: a scalar
// load, that does not wait for the vector loads in front of it.
template <typename V>
__device__ __forceinline__ V scalar_at(const V* p, int64_t i) {
    return *(const __attribute__((address_space(4))) V*)(uintptr_t)(p + i);
}

// The sequence of row t, -1 for a row in front of the first or behind the last.
__device__ __forceinline__ int sequence_of_rows(const LogitArgs& a, int64_t t) {
    if (t >= scalar_at(a.query_start, a.seqs)) return -1;
    return last_low(a.seqs, [&](int j) { return a.query_start[j] <= t; });
}

// The largest of the wave: within rows of 16 lanes, then over the rows, in lane 63 (a
// lane without a partner takes 0).
template <int CTRL>
__device__ __forceinline__ uint32_t max_from(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_from<0x111>(v);  // row_shr 1, 2, 4, 8
    v = max_from<0x112>(v);
    v = max_from<0x114>(v);
    v = max_from<0x118>(v);
    v = max_from<0x142>(v);  // row_bcast 15, 31
    v = max_from<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// The largest key of the wave, as a scalar.
__device__ __forceinline__ uint64_t wave_top(uint64_t key) {
    const uint32_t high = wave_max((uint32_t)(key >> 32));
    const uint32_t low = wave_max((uint32_t)(key >> 32) == high ? (uint32_t)key : 0u);
    return ((uint64_t)high << 32) | low;
}

// A value that all lanes have, in scalar registers.
__device__ __forceinline__ double uniform(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// A load from a scalar address and a lane's offset in bytes.
template <typename V>
__device__ __forceinline__ V load_at(const void* base, uint32_t offset) {
    return *reinterpret_cast<const V*>(static_cast<const char*>(base) + offset);
}

// Threads T, NQ quads a thread: quad k of thread i holds the slice's logits 4 (T k + i) .. .
// LISTS: there is a history, drafted tokens or biases.
template <typename E, int T, int NQ, bool LISTS>
__global__ void __launch_bounds__(T) k_logits(const LogitArgs a) {
    constexpr int kSlice = 4 * T * NQ;
    extern __shared__ uint32_t count[];  // of the slice's tokens (LISTS); then places of their biases
    __shared__ uint64_t sh[kKeys];
    typedef int32_t i4 __attribute__((ext_vector_type(4), aligned(4)));
    const int lo = (int)blockIdx.x * kSlice, size = min(kSlice, (int)a.vocab - lo);
    const bool full = size == kSlice;  // (the last slice of a row goes element by element)
    for (int t = blockIdx.y; t < (int)a.rows; t += gridDim.y) {
        int thread = threadIdx.x;
        asm volatile("" : "+v"(thread));  // made anew: what is computed from it would be held through the loop
        // The row's sequence, its lengths and penalties come by scalar loads, side by side, and
        // a search among sequences before the logits are requested: a vector load waits for
        // those in front of it.
        int seq = t, first = t, n = 1;
        if (a.query_start) {
            seq = __builtin_amdgcn_readfirstlane(sequence_of_rows(a, t));
            if (seq < 0) continue;  // the same for the whole workgroup
        }
        const char* row = a.logits + (t * a.row_stride + lo) * E::bytes;
        float x[NQ][4];
        if (full) {
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
                const auto q = load_at<typename Quad<E>::type>(row, (uint32_t)(4 * (T * k + thread)) * E::bytes);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[k][e] = (float)q[e];
            }
        } else {
#pragma unroll
            for (int k = 0; k < NQ; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int v = 4 * (T * k + thread) + e;
                    const float y = (float)load_at<typename E::elem>(row, (uint32_t)min(v, size - 1) * E::bytes);
                    x[k][e] = v < size ? y : not_a_number();
                }
        }
        int64_t grammar = t;
        if (a.allowed_row) grammar = scalar_at(a.allowed_row, t);
        float repetition = 1.0f, presence = 0.0f, frequency = 0.0f;
        int len = 0, prompt = 0, bias0 = 0, bias1 = 0;
        if constexpr (LISTS) {
            if (a.query_start) {
                first = scalar_at(a.query_start, seq);
                n = scalar_at(a.query_start, seq + 1);
            }
            if (a.history) len = scalar_at(a.history_len, seq);
            if (a.prompt_len) prompt = scalar_at(a.prompt_len, seq);
            if (a.bias_start) {
                bias0 = scalar_at(a.bias_start, seq);
                bias1 = scalar_at(a.bias_start, seq + 1);
            }
            if (a.repetition) repetition = scalar_at(a.repetition, seq);
            if (a.presence) presence = scalar_at(a.presence, seq);
            if (a.frequency) frequency = scalar_at(a.frequency, seq);
            asm volatile("" : "+s"(len), "+s"(prompt), "+s"(bias0), "+s"(bias1), "+s"(first), "+s"(n));  // all at once
            if (a.query_start) n -= first;
            len = min(len, a.history_tokens);
            bias0 = (int)min(max((int64_t)bias0, (int64_t)0), a.biases);
            bias1 = (int)min(max((int64_t)bias1, (int64_t)bias0), a.biases);
        }
        // what is allowed: the words of this thread's logits, used last
        uint32_t open[NQ];
#pragma unroll
        for (int k = 0; k < NQ; ++k) open[k] = ~0u;
        if (a.allowed && grammar >= 0 && grammar < a.allowed_rows) {
            const uint32_t* allowed = a.allowed + grammar * a.allowed_stride + (lo >> 5);
#pragma unroll
            for (int k = 0; k < NQ; ++k) open[k] = load_at<uint32_t>(allowed, 4u * ((uint32_t)min(4 * (T * k + thread), size - 1) >> 5));
        }
        if constexpr (LISTS) {
            // The first round of every list is requested before any is waited for.
            const int32_t* text = a.history + seq * a.history_stride;
            auto tokens_at = [&](int i) {  // four from entry i on, -1 behind the last
                i4 x = {-1, -1, -1, -1};
                if (i + 4 <= len)
                    x = load_at<i4>(text, 4u * (uint32_t)i);
                else
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (i + e < len) x[e] = load_at<int32_t>(text, 4u * (uint32_t)(i + e));
                return x;
            };
            const i4 some = tokens_at(4 * thread);
            // (rows that are not the call's, as wrong starts could name, have no drafts)
            const int own = t - first, most = !a.draft || first < 0 ? 0 : (int)min((int64_t)(a.mask ? min(n, 64 * a.mask_words) : own + 1), a.rows - first);
            const int32_t* draft = a.draft + max(first, 0);
            const uint64_t* mask = a.mask ? a.mask + (int64_t)t * a.mask_words : nullptr;
            auto drafted_at = [&](int j) {  // the j-th drafted token if the row sees it, else -1
                int v = -1;
                if (j < most) {
                    const uint64_t word = mask ? load_at<uint64_t>(mask, 8u * ((uint32_t)j >> 6)) : ~uint64_t(0);
                    v = load_at<int32_t>(draft, 4u * (uint32_t)j);
                    if (!((word >> (j & 63)) & 1)) v = -1;
                }
                return v;
            };
            const int32_t* bias_tokens = a.bias_tokens + bias0;
            const float* bias_values = a.bias_values + bias0;
            const int biases = bias1 - bias0;
            const int drafted = drafted_at(thread);
            const int biased = thread < biases ? load_at<int32_t>(bias_tokens, 4u * (uint32_t)thread) : -1;
            const float value = thread < biases ? load_at<float>(bias_values, 4u * (uint32_t)thread) : 0.0f;
#pragma unroll
            for (int k = 0; k < NQ; ++k) *reinterpret_cast<u4*>(&count[4 * (T * k + thread)]) = u4{0, 0, 0, 0};
            __syncthreads();
            auto note = [&](int token, bool answer) {
                const uint32_t v = (uint32_t)(token - lo);
                if (token < 0 || v >= (uint32_t)size) return;
                if (answer)
                    atomicAdd(&count[v], 1u);
                else
                    atomicOr(&count[v], kPrompt);
            };
            i4 now = some;
            for (int i = 4 * thread; i < len;) {
                const int next = i + 4 * T;
                const i4 then = tokens_at(next);
#pragma unroll
                for (int e = 0; e < 4; ++e) note(now[e], i + e >= prompt);
                now = then;
                i = next;
            }
            note(drafted, true);
            for (int j = T + thread; j < most; j += T) note(drafted_at(j), true);
            __syncthreads();
            // y / repetition from binary64: 1 / repetition and the product are within 2^-52 of the
            // quotient, which is 2^-49 or more from the middle between two binary32 numbers of 24
            // bits, so it is rounded as the quotient is.  (Those of fewer bits are divided.)
            const double inverse = uniform(1.0 / (double)repetition);
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
                u4* place = reinterpret_cast<u4*>(&count[4 * (T * k + thread)]);
                const u4 c4 = *place;
                if (biases > 0) *place = u4{kNoBias, kNoBias, kNoBias, kNoBias};
                if (c4.x | c4.y | c4.z | c4.w) {
                    float y[4];
                    bool small = false;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = x[k][e], q = (float)((double)z * inverse);
                        y[e] = z > 0.0f ? q : z * repetition;
                        small = small || (z > 0.0f && q < 0x1p-125f);
                    }
                    if (small)
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = x[k][e] > 0.0f ? x[k][e] / repetition : y[e];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t answers = c4[e] & ~kPrompt;
                        const float z = rounded(y[e]) - rounded(frequency * (float)answers);
                        x[k][e] = !c4[e] ? x[k][e] : answers ? z - presence : z;
                    }
                }
            }
            if (biases > 0) {
                __syncthreads();
                int* cell = reinterpret_cast<int*>(count);  // kNoBias, or a bias's place
                auto in_slice = [&](int token) { return token >= 0 && (uint32_t)(token - lo) < (uint32_t)size; };
                if (in_slice(biased)) atomicMax(&cell[biased - lo], thread);
                for (int i = T + thread; i < biases; i += T) {
                    const int token = load_at<int32_t>(bias_tokens, 4u * (uint32_t)i);
                    if (in_slice(token)) atomicMax(&cell[token - lo], i);
                }
                __syncthreads();
                if (biases <= T) {  // each has its value at hand: into its cell, if it is the last of its token
                    const bool last = in_slice(biased) && cell[biased - lo] == thread;
                    __syncthreads();
                    if (last) cell[biased - lo] = __builtin_bit_cast(int, value);
                    __syncthreads();
                }
#pragma unroll
                for (int k = 0; k < NQ; ++k) {
                    u4 p4 = *reinterpret_cast<const u4*>(&count[4 * (T * k + thread)]);
                    if (biases > T)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (p4[e] != kNoBias) p4[e] = load_at<uint32_t>(bias_values, 4u * p4[e]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[k][e] = x[k][e] + __builtin_bit_cast(float, (uint32_t)p4[e]);
                }
            }
        }
        float best = none();
        int at = 0;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int v = 4 * (T * k + thread);
            const uint32_t may = open[k] >> (v & 31);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = (may >> e) & 1 ? x[k][e] : none();
                x[k][e] = y;
                if (y > best) {  // (what is behind the slice is NaN, or not allowed)
                    best = y;
                    at = v + e;
                }
            }
        }
        if (a.out) {
            char* dst = reinterpret_cast<char*>(a.out + t * a.out_stride + lo);
            if (full) {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
                    *reinterpret_cast<Quad<F32>::type*>(dst + (uint32_t)(16 * (T * k + thread))) = Quad<F32>::type{x[k][0], x[k][1], x[k][2], x[k][3]};
            } else {
#pragma unroll
                for (int k = 0; k < NQ; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * (T * k + thread) + e < size) *reinterpret_cast<float*>(dst + (uint32_t)(4 * (4 * (T * k + thread) + e))) = x[k][e];
            }
        }
        const uint64_t key = wave_top(best > none() ? argmax_key(best, lo + at) : 0);
        static_assert(T == 64 * kKeys, "a key a wave");
        if (a.slices > 1) {
            if ((thread & 63) == 0) a.keys[(t * a.slices + blockIdx.x) * kKeys + (thread >> 6)] = key;
        } else {
            if ((thread & 63) == 0) sh[thread >> 6] = key;
            __syncthreads();
            uint64_t top = 0;
#pragma unroll
            for (int w = 0; w < kKeys; ++w) top = sh[w] > top ? sh[w] : top;
            if (thread == 0) a.tokens[t] = token_of(top);
        }
        if (t + (int)gridDim.y < (int)a.rows) __syncthreads();  // counts and sh are read before the next row's
    }
}

// tokens[t] from the keys of row t's slices, a wave a row.
__global__ void __launch_bounds__(kThreads) k_logits_pick(const LogitArgs a) {
    constexpr int kAhead = 10;  // 80 slices: one row of 151936
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); t < a.rows; t += (int64_t)gridDim.x * (kThreads / 64)) {
        if (a.query_start && (t < a.query_start[0] || t >= a.query_start[a.seqs])) continue;
        uint64_t best = 0;
        const int total = (int)a.slices * kKeys;
        const uint64_t* keys = a.keys + t * total;
        for (int s = lane; s < total; s += 64 * kAhead) {
            uint64_t v[kAhead];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) v[e] = keys[min(s + 64 * e, total - 1)];
#pragma unroll
            for (int e = 0; e < kAhead; ++e) best = v[e] > best ? v[e] : best;
        }
        best = wave_max_u64(best);
        if (lane == 0) a.tokens[t] = token_of(best);
    }
}

template <typename E, int T, int NQ, bool LISTS>
hipError_t launch(const LogitArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)a.slices, (unsigned)std::min<int64_t>(a.rows, 65535));
    hipLaunchKernelGGL((k_logits<E, T, NQ, LISTS>), grid, dim3(T), LISTS ? 16 * T * NQ : 0, s, a);
    if (a.slices > 1) {
        const unsigned waves = kThreads / 64;
        hipLaunchKernelGGL(k_logits_pick, dim3((unsigned)std::min<int64_t>((a.rows + waves - 1) / waves, 1 << 20)), dim3(kThreads), 0, s, a);
    }
    return hipGetLastError();
}

template <typename E>
hipError_t launch_type(const LogitArgs& a, hipStream_t s) {
    const bool lists = a.history || a.draft || a.bias_start;
    switch (logit_slice(a.rows, a.vocab)) {
        case 2048: return lists ? launch<E, 512, 1, true>(a, s) : launch<E, 512, 1, false>(a, s);
        case 4096: return lists ? launch<E, 512, 2, true>(a, s) : launch<E, 512, 2, false>(a, s);
        default: return lists ? launch<E, 512, 4, true>(a, s) : launch<E, 512, 4, false>(a, s);
    }
}

}  // namespace

// The shortest slice with which the call has no more than two workgroups a CU, 8192 if
// none: few rows end sooner in short slices (one row of 151936: kernel 5.4 us in slices
// of 2048, 6.8 of 8192), many pay for each slice's scan of the history (37 rows of trees
// 23 against 15 us, 192 rows of 4096 tokens 124 against 66).
int64_t logit_slice(int64_t rows, int64_t vocab) {
    int64_t slice = kLogitShort;
    while (slice < kLogitLong && rows * ((vocab + slice - 1) / slice) > kLogitFew) slice *= 2;
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

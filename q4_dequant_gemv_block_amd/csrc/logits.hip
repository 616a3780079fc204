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
// slices' keys (argmax_key) are joined by a second launch, a wave a row; joining in the
// first one would need counters that are zero before every call.
//
// Bound by memory in large batches: 192 rows of 151936 binary32 logits, each with up to
// 4096 tokens and 300 biases, read and written in 62 us of kernel time (3.8 TB/s; a
// large copy reaches 4.7).  Bound by latency in small ones: the sequence, its lengths,
// the lists, the biases' values and the grammar follow each other, 5 us for one row, 13
// for 37 rows of trees, and 2 for the second launch.
#include "kv_device.h"
#include "step_launch.h"
#include "q4gemv.h"

#include <algorithm>

namespace q4 {

namespace {

constexpr int kThreads = 256;  // of the pick
constexpr uint32_t kPrompt = 0x80000000u;

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

// The sequence of row t, -1 for a row in front of the first or behind the last.
__device__ __forceinline__ int sequence_of_rows(const LogitArgs& a, int64_t t) {
    if (t >= a.query_start[a.seqs]) return -1;
    return last_low(a.seqs, [&](int j) { return a.query_start[j] <= t; });
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
    __shared__ uint64_t sh[T / 64];
    typedef int32_t i4 __attribute__((ext_vector_type(4), aligned(4)));
    const int lo = (int)blockIdx.x * kSlice, size = min(kSlice, (int)a.vocab - lo);
    const bool full = size == kSlice;  // (the last slice of a row goes element by element)
    for (int t = blockIdx.y; t < (int)a.rows; t += gridDim.y) {
        int thread = threadIdx.x;
        asm volatile("" : "+v"(thread));  // made anew: what is computed from it would be held through the loop
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
        // the row's sequence, as scalars: what is read by it comes by scalar loads
        int seq = t, first = t, n = 1;
        if (a.query_start) {
            seq = __builtin_amdgcn_readfirstlane(sequence_of_rows(a, t));
            if (seq < 0) continue;  // the same for the whole workgroup
            first = a.query_start[seq];
            n = a.query_start[seq + 1] - first;
        }
        float repetition = 1.0f, presence = 0.0f, frequency = 0.0f;
        if (a.repetition) repetition = a.repetition[seq];
        if (a.presence) presence = a.presence[seq];
        if (a.frequency) frequency = a.frequency[seq];
        int bias0 = 0, bias1 = 0;
        if constexpr (LISTS) {
            int len = 0, prompt = 0;
            if (a.history) {
                len = min(a.history_len[seq], a.history_tokens);
                if (a.prompt_len) prompt = a.prompt_len[seq];
            }
            if (a.bias_start) {
                bias0 = (int)min(max((int64_t)a.bias_start[seq], (int64_t)0), a.biases);
                bias1 = (int)min(max((int64_t)a.bias_start[seq + 1], (int64_t)bias0), a.biases);
            }
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
#pragma unroll
            for (int k = 0; k < NQ; ++k) {
                const int v = 4 * (T * k + thread);
                u4* place = reinterpret_cast<u4*>(&count[v]);
                const u4 c4 = *place;
                if (c4.x | c4.y | c4.z | c4.w) {
                    *place = u4{0, 0, 0, 0};  // (for the biases)
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
            }
            if (biases > 0) {
                __syncthreads();
                auto note_bias = [&](int i, int token) {
                    const uint32_t v = (uint32_t)(token - lo);
                    if (token >= 0 && v < (uint32_t)size) atomicMax(&count[v], (uint32_t)i + 1u);
                };
                note_bias(thread, biased);
                for (int i = T + thread; i < biases; i += T) note_bias(i, load_at<int32_t>(bias_tokens, 4u * (uint32_t)i));
                __syncthreads();
#pragma unroll
                for (int k = 0; k < NQ; ++k) {
                    const u4 p4 = *reinterpret_cast<const u4*>(&count[4 * (T * k + thread)]);
                    if (p4.x | p4.y | p4.z | p4.w) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (p4[e]) x[k][e] = x[k][e] + load_at<float>(bias_values, 4u * (p4[e] - 1u));
                    }
                }
            }
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
            const int v = 4 * (T * k + thread);
            const uint32_t open = allowed ? load_at<uint32_t>(allowed, 4u * ((uint32_t)min(v, size - 1) >> 5)) >> (v & 31) : 15u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = (open >> e) & 1 ? x[k][e] : none();
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
        const uint64_t key = best > none() ? argmax_key(best, lo + at) : 0;
        const uint64_t top = block_max_u64(key, sh);
        if (threadIdx.x == 0) {
            if (a.slices == 1)
                a.tokens[t] = token_of(top);
            else
                a.keys[t * a.slices + blockIdx.x] = top;
        }
        __syncthreads();  // counts and sh are read before the next slice's
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
    int64_t slice = 2048;
    while (slice < 8192 && rows * ((vocab + slice - 1) / slice) > 512) slice *= 2;
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

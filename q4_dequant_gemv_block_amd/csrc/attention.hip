// Attention of a chunk of new tokens over a paged key/value cache (gfx950).
//
// For every new token t and query head h:  out = sum_j p_j v_j / sum_j p_j with
// p_j = exp(scale q.k_j - m) over the keys j the token sees.
//
// Items.  The query heads of a kv head read the same keys, so the rows (token,
// head of the group) of one sequence and kv head are packed into items of 16 NR
// rows (16 or 32); an item's keys are cut into units, and the units of all items, in
// order, are dealt to the workgroups in equal contiguous ranges (ragged
// contexts balance by themselves; the lengths are read on the device).  A range
// that covers an item's keys whole writes its rows; one that holds a part of
// them writes the part's sums, maxima and unnormalised outputs in 32 bits, and
// a second launch joins the parts.
//
// A wave takes 32 keys at a time, straight from HBM into its own part of LDS
// (global_load_lds, whole rows, 16 bytes a lane), so that waves never wait for each
// other: while it works on V, the next step's K is on its way into the place that
// K left, and the next V follows into V's.  (Before the scores the compiler waits
// for the queries in every step, as it does not count on the wait before the loop;
// loads return in order, so V is waited for there too, and only the K of the next
// step is on its way beside work.)
//   S^T = K Q^T on v_mfma_f32_16x16x32, 16 keys a tile: lane (q, n) gets the keys 4 q
//     .. 4 q + 3 of both tiles for query row n, which is the B operand P^T of
//   O^T = V^T P^T, whose A operand the transposing LDS reads give for the same keys.
// Rows lie in LDS as long as a head, their 16-byte chunks XORed by the row so that
// the reads of both products use all 64 banks.  Loading to registers instead, K in
// the operand's layout (half lines of 16 rows a load), took 2.4 us for a step of 8
// waves on a CU, this 1.6.
// The loads are non-temporal: each 128-byte line is used once.
// The reference m of a row's weights is raised only when a score exceeds the one it
// was made from by 2^8 (kLift in attn_device.h), so most steps neither reduce over
// lanes nor rescale.  Row sums are of the rounded probabilities, so
// a rounding does not shift a row's weight.
//
// Bound by HBM.  Measured, 32 query heads over 8 of 128: 61 ragged sequences up to
// 8192 keys 180 us and 5 for the join (6.4 TB/s; a read alone reaches 7.2 on this
// card), one token over 131067 keys 84 and 5 (6.4 TB/s); one token over 515 keys of
// 40 heads 8.7, the latency of 3 steps.
#include "attn_device.h"
#include "attn_shape.h"
#include "q4gemv.h"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace q4 {

namespace {

constexpr int kThreads = 256;     // of a joining workgroup
constexpr int kStep = kAttnStep;  // keys of one step of a wave

template <typename T>
struct Mma;
template <>
struct Mma<F16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};
template <>
struct Mma<BF16> {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f4 mma(u4 a, u4 b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};

// Waves of a workgroup of k_attn, one workgroup a CU: as many as 128 KiB of LDS
// hold 32 keys of K and V for.
constexpr int attn_waves(int head_dim) { return head_dim <= 128 ? 8 : 4; }

// Places in LDS: a wave's 32 rows of K, then as many of V.
template <int D, int NR>
struct Layout : LdsRow<D> {
    typedef LdsRow<D> R;
    static constexpr int loads = kStep / R::per_load;     // of K, and of V, a step
    static constexpr int bytes = kStep * R::row;
    static constexpr int waves = attn_waves(D);
    static constexpr int lines = D + 4;                   // floats of a row of outputs
    // after the keys, in their place: outputs of all waves, their maxima and sums
    static constexpr int merge = waves * 16 * NR * (lines + 2) * 4;
    static constexpr int total = merge > 2 * waves * bytes ? merge : 2 * waves * bytes;
    // V's transposing reads take 32 bytes of 8 rows at a time
    static __device__ __forceinline__ int swz_v(int r) { return R::chunks == 8 ? ((r >> 1) & 3) << 1 : (r & 7) << 1; }
};

template <typename T, int D, int NR, typename WORK>
__global__ void __launch_bounds__(attn_waves(D) * 64) k_attn(const AttnArgs a, const Cut cut) {
    typedef Layout<D, NR> L;
    constexpr int ROWS = 16 * NR, kWaves = L::waves;
    constexpr int KS = D / 32;  // k-steps of the first product
    constexpr int DT = D / 16;  // 16-element tiles of the output
    extern __shared__ char sh[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, n16 = lane & 15;
    WORK work;
    Item it;
    if (!work.start(cut, a.batch, &it)) return;
    const Seq& seq = work.seq;
    const Parts<D> parts(a.workspace, (int)gridDim.x, ROWS);
    // this wave's K and V, and where the lane reads in them
    char* my = sh + wave * 2 * L::bytes;
    const uint32_t my_lds = lds_address(my);
    const char* at_k = my + n16 * L::row;
    const int chunk_k = q ^ L::swz_k(n16);
    const int row_v = 4 * q + (n16 >> 2);
    const char* at_v = my + L::bytes + row_v * L::row + (n16 & 1) * 8;
    const int chunk_v = ((n16 & 3) >> 1) ^ L::swz_v(row_v);
    const bool one_page = a.cache.page_size.d % kStep == 0;  // a step's keys lie in one page
    while (work.next(cut, a.batch, &it)) {
        const int head = it.head, row0 = it.row0, rows = it.rows, past = it.past;
        const int p_first = it.p_first, p_last = it.p_last, k_lo = it.k_lo, k_hi = it.k_hi;

        // queries: B operands, rows n16 of each 16-row tile
        u4 qf[NR][KS];
        int pos[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = row0 + 16 * r + n16;
            const int rc = min(row, row0 + rows - 1);
            const int i = (int)cut.group.div(rc), h = head * a.group + rc - i * a.group;
            pos[r] = row < row0 + rows ? past + i : -1;
            const char* src = a.q.data + ((int64_t)(seq.row0 + i) * a.q.token_stride + (int64_t)h * a.q.head_stride + 8 * q) * 2;
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[r][s] = *reinterpret_cast<const u4*>(src + 64 * s);
        }
        f4 acc[NR][DT];
        float m[NR], l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = kNone;
            l[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < DT; ++j) acc[r][j] = f4{0, 0, 0, 0};
        }
        // (no kernel of the call writes the table: constant, and so read by scalar loads)
        typedef const __attribute__((address_space(4))) int32_t c_i32;
        c_i32* table = (c_i32*)(uintptr_t)(a.batch.table + seq.b * a.batch.table_stride);
        const char* kbase = a.cache.k + (int64_t)head * a.cache.k_head * 2;
        const char* vbase = a.cache.v + (int64_t)head * a.cache.v_head * 2;

        // The pages of a step's four groups of 8 keys (scalar loads: a wait for
        // them does not wait for the keys on their way).
        struct Pages {
            int p[4];
        };
        auto pages = [&](int t) {
            Pages x;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t column = a.cache.page_size.div((uint32_t)(t + 8 * g));
                const int page = table[min(column, (uint32_t)a.batch.table_pages - 1)];
                x.p[g] = column < (uint32_t)a.batch.table_pages && (uint32_t)page < a.cache.pages ? page : -1;
                if (one_page) {
                    x.p[1] = x.p[2] = x.p[3] = x.p[0];
                    break;
                }
            }
            return x;
        };
        auto fill = [&](int t, const Pages& x, const char* base, int64_t page_stride, int64_t slot_stride, uint32_t to, bool values) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t p = (uint32_t)(t + 8 * g);
                const uint32_t slot = p - a.cache.page_size.div(p) * a.cache.page_size.d;
                const char* src = base + ((int64_t)max(x.p[g], 0) * page_stride + (int64_t)slot * slot_stride) * 2;
#pragma unroll
                for (int k = 0; k < L::loads / 4; ++k) {
                    const int r8 = k * L::per_load + lane / L::chunks, r = 8 * g + r8;
                    const int c = (lane % L::chunks) ^ (values ? L::swz_v(r) : L::swz_k(r));
                    if (D == 8 * L::chunks || c < D / 8)
                        load_to_lds_once(src, r8 * (uint32_t)slot_stride * 2 + 16 * c, to + (8 * g + k * L::per_load) * L::row);
                }
            }
        };
        auto fill_k = [&](int t, const Pages& x) { fill(t, x, kbase, a.cache.k_page, a.cache.k_slot, my_lds, false); };
        auto fill_v = [&](int t, const Pages& x) { fill(t, x, vbase, a.cache.v_page, a.cache.v_slot, my_lds + L::bytes, true); };

        int t = k_lo + wave * kStep;
        Pages now = {}, next = {};
        if (t < k_hi) now = pages(t);
        __builtin_amdgcn_s_waitcnt(0x0F70);  // the queries
        if (t < k_hi) {
            fill_k(t, now);
            fill_v(t, now);
            next = pages(t + kWaves * kStep);
        }
        for (; t < k_hi; t += kWaves * kStep) {
            const int t_next = t + kWaves * kStep;
            const bool more = t_next < k_hi;
            // S^T: keys 4 q + j and 16 + 4 q + j in the lane's query rows
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L::loads) : "memory");  // K is there, V on its way
            float s[NR][8];
            {
                u4 kf[2][KS];
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u) kf[u][k] = *reinterpret_cast<const u4*>(at_k + ((chunk_k ^ (4 * k)) * 16) + u * 16 * L::row);
                __builtin_amdgcn_sched_barrier(0);  // all reads before the products
                f4 c[NR][2];
#pragma unroll
                for (int r = 0; r < NR; ++r) c[r][0] = c[r][1] = f4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < NR; ++r) c[r][u] = Mma<T>::mma(kf[u][k], qf[r][k], c[r][u]);
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[r][j] = c[r][j >> 2][j & 3];
            }
            const Pages here = now;
            if (more) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // K is read
                fill_k(t_next, next);
                now = next;
                next = pages(t_next + kWaves * kStep);
            }
            // masks: only steps that some row does not see whole
            uint32_t valid = 0;  // groups with a place
#pragma unroll
            for (int g = 0; g < 4; ++g) valid |= (here.p[g] >= 0 ? 1u : 0u) << g;
            const bool ragged = t + kStep > min(k_hi, p_first + 1) || (a.window && t <= p_last - a.window) || valid != 15;
            uint32_t places = 0xFFFFFFFFu;  // keys of the step that are there
            if (ragged) {
                places = (uint32_t)bits_between(0, k_hi - t);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (!((valid >> g) & 1)) places &= ~(0xFFu << (8 * g));
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint32_t seen = places & (uint32_t)bits_between(a.window ? pos[r] - a.window + 1 - t : 0, pos[r] + 1 - t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[r][j] = keep_seen(s[r][j], bit_mask(seen >> (4 * q), 16 * (j >> 2) + (j & 3)));
                }
            }
            uint32_t p[NR][4];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float top = s[r][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top = fmaxf(top, s[r][j]);
                top *= a.scale_log2;
                if (__ballot(top > m[r] + kRaise<T>)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float raised = top > m[r] + kRaise<T> ? top - kLift<T> : m[r];  // each row by itself
                    const float f = raised == kNone ? 1.0f : __builtin_amdgcn_exp2f(m[r] - raised);
                    m[r] = raised;
                    l[r] *= f;
#pragma unroll
                    for (int j = 0; j < DT; ++j) acc[r][j] *= f;
                }
                const float ref = m[r] == kNone ? 0.0f : m[r];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][2 * j], a.scale_log2, -ref));
                    const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][2 * j + 1], a.scale_log2, -ref));
                    p[r][j] = pack2<T>(e0, e1);
                    l[r] = add_pair<T>(p[r][j], l[r]);
                }
            }
            if (more)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L::loads) : "memory");  // V is there, the next K on its way
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (ragged) {
                // Values of keys that do not belong here become 0.  So do NaN and
                // infinities - in a product a weight of 0 times them would reach
                // rows that do not see the key - and are added row by row to
                // those that do.
                uint32_t any = 0;
#pragma unroll
                for (int k = 0; k < L::loads; ++k) {
                    const int r = k * L::per_load + lane / L::chunks;
                    u4* at = reinterpret_cast<u4*>(my + L::bytes + k * 1024 + lane * 16);
                    const int c = (lane % L::chunks) ^ L::swz_v(r);
                    if (D != 8 * L::chunks && c >= D / 8) continue;
                    const u4 v = *at;
                    const uint32_t keep = bit_mask(places >> (r & 31), 0);
                    const u4 bad = {nonfinite<T>(v.x), nonfinite<T>(v.y), nonfinite<T>(v.z), nonfinite<T>(v.w)};
                    any |= (bad.x | bad.y | bad.z | bad.w) & keep;
                    *at = v & ~bad & keep;
                }
                wave_lds_fence();
                if (__ballot(any != 0)) {
                    for (int k = 0; k < kStep; ++k) {
                        if (!((places >> k) & 1)) continue;
                        const int page = k < 16 ? (k < 8 ? here.p[0] : here.p[1]) : (k < 24 ? here.p[2] : here.p[3]);
                        const uint32_t slot = (uint32_t)(t + k) - a.cache.page_size.div(t + k) * a.cache.page_size.d;
                        const char* src = vbase + ((int64_t)page * a.cache.v_page + (int64_t)slot * a.cache.v_slot + 4 * q) * 2;
                        float w[NR];
                        bool sees[NR];
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            uint32_t pr = 0;  // keys 16 (j / 2) + 4 q + 2 (j % 2), + 1
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if ((k & ~13) == 16 * (j >> 1) + 2 * (j & 1)) pr = p[r][j];
                            w[r] = half_of<T>((uint32_t)__shfl((int)pr, n16 + 16 * ((k >> 2) & 3)), k & 1);
                            sees[r] = t + k <= pos[r] && (!a.window || t + k > pos[r] - a.window);
                        }
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            float v[4];
                            load_elems<T, 4>(src + 32 * d, v);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int r = 0; r < NR; ++r)
                                    if (sees[r] && !__builtin_isfinite(v[i])) acc[r][d][i] += w[r] * v[i];
                            __builtin_amdgcn_sched_barrier(0);  // registers: one load at a time
                        }
                    }
                }
            }
            // O^T += V^T P^T
            constexpr int HALF = DT / 2;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                u4 vf[HALF];
#pragma unroll
                for (int d = 0; d < HALF; ++d) {
                    const char* src = at_v + ((chunk_v ^ (2 * (b * HALF + d))) * 16);
                    vf[d] = read_transposed(src, src + 16 * L::row);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int d = 0; d < HALF; ++d)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        acc[r][b * HALF + d] = Mma<T>::mma(vf[d], u4{p[r][0], p[r][1], p[r][2], p[r][3]}, acc[r][b * HALF + d]);
            }
            if (more) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // V is read
                fill_v(t_next, now);
            }
        }

        // the waves' sums: elements 16 d + 4 q .. of row n16, in the place of the keys
        __syncthreads();
        float* sh_o = reinterpret_cast<float*>(sh);
        float* sh_m = sh_o + kWaves * ROWS * L::lines;
        float* sh_l = sh_m + kWaves * ROWS;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            l[r] += __shfl_xor(l[r], 16);
            l[r] += __shfl_xor(l[r], 32);
            const int at = wave * ROWS + 16 * r + n16;
            if (q == 0) {
                sh_m[at] = m[r];
                sh_l[at] = l[r];
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) *reinterpret_cast<f4*>(&sh_o[at * L::lines + 16 * d + 4 * q]) = acc[r][d];
        }
        __syncthreads();
        const bool whole = work.whole(it);
        const int64_t slot = (int64_t)2 * blockIdx.x + (it.u0 == 0);
        for (int u = threadIdx.x; u < rows * (D / 4); u += 64 * kWaves) {
            const int row = u / (D / 4), d = (u - row * (D / 4)) * 4;
            float top = kNone;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sh_m[w * ROWS + row]);
            const float ref = top == kNone ? 0.0f : top;
            f4 o = {0, 0, 0, 0};
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(sh_m[w * ROWS + row] - ref);
                sum += f * sh_l[w * ROWS + row];
                o += f * *reinterpret_cast<const f4*>(&sh_o[(w * ROWS + row) * L::lines + d]);
            }
            if (whole) {
                const float f = row_scale(sum);
                const int i = (int)cut.group.div(row0 + row), h = head * a.group + row0 + row - i * a.group;
                float v[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
                store_elems<T, 4>(a.out.data + ((int64_t)(seq.row0 + i) * a.out.token_stride + (int64_t)h * a.out.head_stride + d) * 2, v);
                if (a.lse && d == 0) a.lse[(int64_t)(seq.row0 + i) * a.q_heads + h] = row_lse(top, sum);
            } else {
                *reinterpret_cast<f4*>(&parts.o[(slot * ROWS + row) * D + d]) = o;
                if (d == 0) parts.ml[slot * ROWS + row] = f2{top, sum};
            }
        }
        if constexpr (WORK::once) break;
        __syncthreads();
    }
}

// Joins the parts of the items that several ranges share.  Workgroup (w, y)
// takes the item that begins in range w and does not end there, if there is
// one, and every gridDim.y-th batch of its rows: one SG-lane group a row where
// the parts are few, all groups on one row where they are many.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_attn_join(const AttnArgs a, const Cut cut, uint32_t slots) {
    constexpr int SG = D <= 64 ? 16 : D <= 128 ? 32 : 64;  // lanes of a row
    constexpr int NSG = kThreads / SG;
    __shared__ f4 sh_o[NSG][SG];
    __shared__ float sh_s[NSG];
    Work work;
    work.sum(cut, a.batch);
    const uint32_t total = work.total, grid = min(slots, total), w0 = blockIdx.x;
    if (w0 + 1 >= grid) return;
    const uint32_t border = range_begin(total, w0 + 1, grid);
    if (!work.find(cut, a.batch, border)) return;
    const Seq& seq = work.seq;
    const uint32_t item = (border - work.begin) / (uint32_t)seq.units;
    const uint32_t first = work.begin + item * seq.units, last = first + seq.units - 1;
    if (first == border || first < range_begin(total, w0, grid) || last >= total) return;
    uint32_t w1 = (uint32_t)((uint64_t)last * grid / total);  // the range that holds `last`
    while (range_begin(total, w1 + 1, grid) <= last) ++w1;
    while (range_begin(total, w1, grid) > last) --w1;
    Item it;
    place_item(cut, seq, item, &it);
    const int R = 1 << cut.rows_log2;
    const Parts<D> parts(a.workspace, (int)slots, R);
    const int g = threadIdx.x / SG, lane = threadIdx.x & (SG - 1), d = lane * 4;
    const bool many = w1 - w0 >= NSG;
    const int stride = many ? 1 : NSG;
    for (int row = blockIdx.y * stride + (many ? 0 : g); row < it.rows; row += gridDim.y * stride) {
        // part of range w: slot 2 w + 1 in the item's first range, else 2 w
        auto slot_of = [&](uint32_t w) { return ((int64_t)2 * w + (w == w0)) * R + row; };
        const uint32_t from = w0 + (many ? g : 0), by = many ? NSG : 1;
        float top = kNone, sum = 0.0f;
        f4 o = {0, 0, 0, 0};
        for (uint32_t w = from; w <= w1; w += 4 * by) {
            f2 ml[4];
            f4 po[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = w + k * by <= w1;
                ml[k] = in ? parts.ml[slot_of(w + k * by)] : f2{kNone, 0.0f};
                po[k] = in && d < D ? *reinterpret_cast<const f4*>(&parts.o[slot_of(w + k * by) * D + d]) : f4{0, 0, 0, 0};
            }
            const float raised = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), top);
            const float ref = raised == kNone ? 0.0f : raised;
            const float keep = __builtin_amdgcn_exp2f(top - ref);
            sum *= keep;
            o *= keep;
            top = raised;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = __builtin_amdgcn_exp2f(ml[k].x - ref);
                sum += f * ml[k].y;
                o += f * po[k];
            }
        }
        if (many) {
            // all groups' sums to the largest maximum, then over the groups
            __shared__ float sh_m[NSG];
            if (lane == 0) sh_m[g] = top;
            __syncthreads();
            float all = sh_m[0];
#pragma unroll
            for (int k = 1; k < NSG; ++k) all = fmaxf(all, sh_m[k]);
            const float f = __builtin_amdgcn_exp2f(top - (all == kNone ? 0.0f : all));
            top = all;
            sh_o[g][lane] = o * f;
            if (lane == 0) sh_s[g] = sum * f;
            __syncthreads();
            if (g == 0) {
                o = sh_o[0][lane];
                sum = sh_s[0];
#pragma unroll
                for (int k = 1; k < NSG; ++k) {
                    o += sh_o[k][lane];
                    sum += sh_s[k];
                }
            }
            __syncthreads();
        }
        if ((!many || g == 0) && d < D) {
            const float f = row_scale(sum);
            const int i = (int)cut.group.div(it.row0 + row), h = it.head * a.group + it.row0 + row - i * a.group;
            float v[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
            store_elems<T, 4>(a.out.data + ((int64_t)(seq.row0 + i) * a.out.token_stride + (int64_t)h * a.out.head_stride + d) * 2, v);
            if (a.lse && d == 0) a.lse[(int64_t)(seq.row0 + i) * a.q_heads + h] = row_lse(top, sum);
        }
    }
}

int compute_units() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

Cut make_cut(const AttnArgs& a, const AttnShape& s) {
    Cut c = {};
    c.rows_log2 = __builtin_ctz(s.rows);
    c.unit_log2 = __builtin_ctz(s.unit);
    c.step = s.step;
    c.window = a.window;
    c.per_token = s.per_token;
    c.group = FastDiv((uint32_t)a.group);
    c.kv_heads = FastDiv((uint32_t)a.cache.kv_heads);
    c.capacity = (int)((int64_t)a.batch.table_pages * a.cache.page_size.d);
    c.tokens = a.tokens;
    return c;
}

template <typename T, int D, int NR, typename WORK>
hipError_t launch_work(const AttnArgs& a, const AttnShape& shape, hipStream_t s) {
    constexpr size_t lds = Layout<D, NR>::total;
    static LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(k_attn<T, D, NR, WORK>), lds);
    if (e != hipSuccess) return e;
    return launch_shape(shape, make_cut(a, shape), [&](unsigned grid, const Cut& c) {
        hipLaunchKernelGGL((k_attn<T, D, NR, WORK>), dim3(grid), dim3(64 * Layout<D, NR>::waves), lds, s, a, c);
    });
}

template <typename T, int D, int NR>
hipError_t launch(const AttnArgs& a, const AttnShape& shape, hipStream_t s) {
    return shape.places ? launch_work<T, D, NR, Places>(a, shape, s) : launch_work<T, D, NR, Work>(a, shape, s);
}

template <typename T, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnShape& shape, hipStream_t s) {
    hipError_t e = hipErrorInvalidValue;
    if (shape.rows >= 64)
        e = launch_attn_tile<T, D>(a, make_cut(a, shape), shape, s);
    else if (shape.rows == 16)
        e = launch<T, D, 1>(a, shape, s);
    else
        e = launch<T, D, 2>(a, shape, s);
    if (e != hipSuccess || !shape.bytes || shape.grid < 2) return e;
    // Few items have many parts each: a workgroup a row; else one for eight rows.
    const int by = std::min(16, shape.few ? shape.most_rows : (shape.most_rows + 7) / 8);
    hipLaunchKernelGGL((k_attn_join<T, D>), dim3((unsigned)shape.grid - 1, by), dim3(kThreads), 0, s, a, make_cut(a, shape), (uint32_t)shape.grid);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_type(const AttnArgs& a, const AttnShape& shape, hipStream_t s) {
    switch (a.cache.head_dim) {
        case 64: return launch_dim<T, 64>(a, shape, s);
        case 96: return launch_dim<T, 96>(a, shape, s);
        case 128: return launch_dim<T, 128>(a, shape, s);
        default: return launch_dim<T, 256>(a, shape, s);
    }
}

}  // namespace

hipError_t LdsLimit::raise(const void* kernel, size_t bytes) {
    if (bytes <= 65536) return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return hipSuccess;
    e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

bool attn_head_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

AttnShape attn_shape(const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int window, int max_query, int max_context) {
    return attn_shape_on(compute_units(), c, b, q_heads, tokens, window, max_query, max_context);
}

hipError_t launch_attention(const AttnArgs& a, const AttnShape& shape, int type, hipStream_t s) {
    return type == Q4_TYPE_F16 ? launch_type<F16>(a, shape, s) : launch_type<BF16>(a, shape, s);
}

}  // namespace q4

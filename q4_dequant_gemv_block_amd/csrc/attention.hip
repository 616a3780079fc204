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
// A wave takes 32 keys at a time from HBM straight into registers, with no LDS
// and no data movement between lanes:
//   S^T = K Q^T on v_mfma_f32_16x16x32: two tiles of 16 keys.  Tile a holds the
//     keys 8 (m / 4) + 4 a + m % 4 in its rows m, so that the lane that gets
//     rows 4 q .. 4 q + 3 of both tiles has the 8 consecutive keys 8 q .. 8 q + 7
//     of one query row - which is the B operand P^T of the second product.
//   O^T = V^T P^T: lane (q, i) reads D/16 consecutive elements of keys 8 q .. 8 q
//     + 7 (16 lanes read a whole row of V), and transposes its 8 x D/16 block by
//     byte permutes into D/16 A operands; row i of operand j is element
//     D/16 i + j.  The accumulators of lane (q, n) are then the consecutive
//     elements D/4 q .. of query row n.
// V's loads are non-temporal: a load takes whole 128-byte lines, once (212 -> 196 us
// for 61 sequences of up to 8192 keys; K's, which take half lines, gain nothing).
// The running maximum is raised only when a score exceeds it by 2^8 (the
// probabilities stay below 2^8, far inside both types), so most steps neither
// reduce over lanes nor rescale.  Row sums are of the rounded probabilities, so
// a rounding does not shift a row's weight.
#include "attn_device.h"
#include "q4gemv.h"

#include <algorithm>
#include <atomic>

namespace q4 {

namespace {

constexpr int kThreads = 256;     // of a joining workgroup
constexpr int kStep = 32;         // keys of one step of a wave

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

// 32 keys of one wave in registers.
template <int D>
struct Keys {
    u4 k[2][D / 32];           // tile a: A operand of k-step s
    uint32_t v[8][D / 32];     // key 8 q + t: elements D/16 i ..
};

// Waves of a workgroup of k_attn, one workgroup a CU: as many as its registers
// allow (two a SIMD, one where 32 rows of 128 or heads of 256 take over 256).
constexpr int attn_waves(int head_dim, int rows) { return head_dim * rows <= 16 * 192 ? 8 : 4; }

template <typename T, int D, int NR>
__global__ void __launch_bounds__(attn_waves(D, 16 * NR) * 64) k_attn(const AttnArgs a, const Cut cut) {
    constexpr int ROWS = 16 * NR, kWaves = attn_waves(D, ROWS), kThreads = 64 * kWaves;
    constexpr int PER = D / 16;      // elements of V a lane holds of a key
    constexpr int KS = D / 32;       // k-steps of the first product
    constexpr int LD = D + 4;
    // [wave][ROWS][LD] outputs, [wave][ROWS] maxima, the same of sums, [wave][ROWS][kStep] weights
    extern __shared__ float sh[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int q = lane >> 4, n16 = lane & 15;
    Work work;
    if (!work.start(cut, a.batch)) return;
    const Seq& seq = work.seq;
    const Parts<D> parts(a.workspace, (int)gridDim.x, ROWS);
    Item it;
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
        f4 acc[NR][PER];
        float m[NR], l[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = kNone;
            l[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < PER; ++j) acc[r][j] = f4{0, 0, 0, 0};
        }
        const int32_t* table = a.batch.table + seq.b * a.batch.table_stride;
        const char* kbase = a.cache.k + (int64_t)head * a.cache.k_head * 2 + 16 * q;
        const char* vbase = a.cache.v + (int64_t)head * a.cache.v_head * 2 + n16 * PER * 2;

        // pages of the two groups of 8 keys this lane reads in the step at key t
        auto pages = [&](int t, int* pk, int* pv) {
            *pk = page_of(a.cache, a.batch, table, t + 8 * (n16 >> 2));
            *pv = page_of(a.cache, a.batch, table, t + 8 * q);
        };
        auto load_k = [&](int t, int page, Keys<D>& x) {
            const uint32_t p = (uint32_t)(t + 8 * (n16 >> 2));
            const uint32_t slot = p - a.cache.page_size.div(p) * a.cache.page_size.d + (n16 & 3);
            const char* src = kbase + ((int64_t)max(page, 0) * a.cache.k_page + (int64_t)slot * a.cache.k_slot) * 2;
#pragma unroll
            for (int t4 = 0; t4 < 2; ++t4)
#pragma unroll
                for (int s = 0; s < KS; ++s) x.k[t4][s] = *(g_u4*)(src + t4 * 8 * a.cache.k_slot + 64 * s);
        };
        auto load_v = [&](int t, int page, Keys<D>& x) {
            const uint32_t p = (uint32_t)(t + 8 * q);
            const uint32_t slot = p - a.cache.page_size.div(p) * a.cache.page_size.d;
            const char* src = vbase + ((int64_t)max(page, 0) * a.cache.v_page + (int64_t)slot * a.cache.v_slot) * 2;
#pragma unroll
            for (int t8 = 0; t8 < 8; ++t8) {
                typedef uint32_t raw __attribute__((ext_vector_type(PER / 2), aligned(4)));
                const raw r = __builtin_nontemporal_load((__attribute__((address_space(1))) const raw*)(src + t8 * 2 * a.cache.v_slot));
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) x.v[t8][j] = r[j];
            }
        };

        Keys<D> x;
        int t = k_lo + wave * kStep;
        int pk, pv, pk_next, pv_next;
        if (t < k_hi) {
            pages(t, &pk, &pv);
            load_k(t, pk, x);
            load_v(t, pv, x);
            pages(t + kWaves * kStep, &pk_next, &pv_next);
        }
        for (; t < k_hi; t += kWaves * kStep) {
            // S^T: scores of keys t + 8 q .. + 7 in the lane's query rows
            float s[NR][8];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int t4 = 0; t4 < 2; ++t4) {
                    f4 c = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < KS; ++k) c = Mma<T>::mma(x.k[t4][k], qf[r][k], c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[r][4 * t4 + j] = c[j];
                }
            const int t_next = t + kWaves * kStep;
            const bool more = t_next < k_hi;
            const int pv_now = pv;
            if (more) {
                load_k(t_next, pk_next, x);
                pv = pv_next;
                pages(t_next + kWaves * kStep, &pk_next, &pv_next);
            }
            // masks: only steps that some row does not see whole
            const bool ragged = t + kStep > min(k_hi, p_first + 1) || (a.window && t <= p_last - a.window) ||
                                __ballot(pv_now < 0) != 0;
            if (ragged) {
                const int first = t + 8 * q;
                // keys that do not belong here: their values could be anything
                const uint32_t here = pv_now < 0 ? 0u : (uint32_t)bits_between(0, k_hi - first);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t mask = bit_mask(here, j);
#pragma unroll
                    for (int e = 0; e < PER / 2; ++e) x.v[j][e] &= mask;
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint32_t seen = here & (uint32_t)bits_between(a.window ? pos[r] - a.window + 1 - first : 0, pos[r] + 1 - first);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[r][j] = keep_seen(s[r][j], bit_mask(seen, j));
                }
            }
            uint32_t p[NR][4];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float top = s[r][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top = fmaxf(top, s[r][j]);
                top *= a.scale_log2;
                if (__ballot(top > m[r] + kRaise)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float raised = top > m[r] + kRaise ? top : m[r];  // each row by itself
                    const float f = raised == kNone ? 1.0f : __builtin_amdgcn_exp2f(m[r] - raised);
                    m[r] = raised;
                    l[r] *= f;
#pragma unroll
                    for (int j = 0; j < PER; ++j) acc[r][j] *= f;
                }
                const float ref = m[r] == kNone ? 0.0f : m[r];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][2 * j], a.scale_log2, -ref));
                    const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][2 * j + 1], a.scale_log2, -ref));
                    p[r][j] = pack2<T>(e0, e1);
                    l[r] += unpack_sum<T>(p[r][j]);
                }
            }
            if (ragged) {
                // In a product a weight of 0 times NaN or infinity would reach
                // rows that do not see the key: such elements leave the
                // product and are added row by row to those that do see them.
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < PER / 2; ++e) any |= nonfinite_bits<T>(x.v[j][e]);
                if (__ballot(any != 0)) {
                    // through this wave's part of LDS: rare, and so free of registers
                    float* so = sh + wave * ROWS * LD;
                    float* sp = sh + kWaves * ROWS * (LD + 2) + wave * ROWS * kStep;
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
#pragma unroll
                        for (int rr = 0; rr < 4; ++rr)
#pragma unroll
                            for (int j = 0; j < PER; ++j) so[(16 * r + n16) * LD + D / 4 * q + PER * rr + j] = acc[r][j][rr];
#pragma unroll
                        for (int j = 0; j < 8; ++j) sp[(16 * r + n16) * kStep + 8 * q + j] = half_of<T>(p[r][j / 2], j & 1);
                    }
                    wave_lds_fence();
                    for (int k = 0; k < kStep && t + k < k_hi; ++k) {
                        const int page = page_of(a.cache, a.batch, table, t + k);
                        if (page < 0) continue;
                        const int64_t at = page * a.cache.v_page + head * a.cache.v_head +
                                           (int64_t)(t + k - (int)a.cache.page_size.div(t + k) * (int)a.cache.page_size.d) * a.cache.v_slot;
                        for (int d = lane; d < D; d += 64) {
                            float v;
                            load_elems<T, 1>(a.cache.v + (at + d) * 2, reinterpret_cast<float(&)[1]>(v));
                            if (__builtin_isfinite(v)) continue;
                            for (int row = 0; row < rows; ++row) {
                                const int pr = past + (int)cut.group.div(row0 + row);
                                if (t + k <= pr && (!a.window || t + k > pr - a.window)) so[row * LD + d] += sp[row * kStep + k] * v;
                            }
                        }
                    }
                    wave_lds_fence();
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int rr = 0; rr < 4; ++rr)
#pragma unroll
                            for (int j = 0; j < PER; ++j) acc[r][j][rr] = so[(16 * r + n16) * LD + D / 4 * q + PER * rr + j];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int e = 0; e < PER / 2; ++e) x.v[j][e] &= ~nonfinite<T>(x.v[j][e]);
                }
            }
            // O^T += V^T P^T: dim pairs (2 e, 2 e + 1) of the 8 keys become two A operands
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) {
                u4 even, odd;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    even[j] = __builtin_amdgcn_perm(x.v[2 * j + 1][e], x.v[2 * j][e], 0x05040100u);
                    odd[j] = __builtin_amdgcn_perm(x.v[2 * j + 1][e], x.v[2 * j][e], 0x07060302u);
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const u4 pb = {p[r][0], p[r][1], p[r][2], p[r][3]};
                    acc[r][2 * e] = Mma<T>::mma(even, pb, acc[r][2 * e]);
                    acc[r][2 * e + 1] = Mma<T>::mma(odd, pb, acc[r][2 * e + 1]);
                }
            }
            if (more) load_v(t_next, pv, x);
        }

        // the four waves' sums: elements D/4 q + PER rr + j of row n16 (rr: accumulator row)
        float* sh_m = sh + kWaves * ROWS * LD;
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
            for (int rr = 0; rr < 4; ++rr)
#pragma unroll
                for (int j = 0; j < PER; ++j) sh[at * LD + D / 4 * q + PER * rr + j] = acc[r][j][rr];
        }
        __syncthreads();
        const bool whole = it.u0 == 0 && it.u1 == seq.units;
        const int64_t slot = (int64_t)2 * blockIdx.x + (it.u0 == 0);
        for (int u = threadIdx.x; u < rows * (D / 4); u += kThreads) {
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
                o += f * *reinterpret_cast<const f4*>(&sh[(w * ROWS + row) * LD + d]);
            }
            if (whole) {
                const float f = row_scale(sum);
                const int i = (int)cut.group.div(row0 + row), h = head * a.group + row0 + row - i * a.group;
                float v[4] = {o.x * f, o.y * f, o.z * f, o.w * f};
                store_elems<T, 4>(a.out.data + ((int64_t)(seq.row0 + i) * a.out.token_stride + (int64_t)h * a.out.head_stride + d) * 2, v);
                if (a.lse && d == 0)
                    a.lse[(int64_t)(seq.row0 + i) * a.q_heads + h] = row_lse(top, sum);
            } else {
                *reinterpret_cast<f4*>(&parts.o[(slot * ROWS + row) * D + d]) = o;
                if (d == 0) parts.ml[slot * ROWS + row] = f2{top, sum};
            }
        }
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
    if (first == border || first < range_begin(total, w0, grid)) return;
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

// Most items a call can have: a sequence's rows round up once.
int64_t item_bound(const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int rows) {
    return (int64_t)c.kv_heads * (tokens * (q_heads / c.kv_heads) / rows + std::min<int64_t>(b.seqs, tokens));
}

Cut make_cut(const AttnArgs& a, const AttnShape& s) {
    Cut c = {};
    c.rows_log2 = __builtin_ctz(s.rows);
    c.unit_log2 = __builtin_ctz(s.unit);
    c.step = s.step;
    c.window = a.window;
    c.group = FastDiv((uint32_t)a.group);
    c.kv_heads = FastDiv((uint32_t)a.cache.kv_heads);
    c.capacity = (int)((int64_t)a.batch.table_pages * a.cache.page_size.d);
    c.tokens = a.tokens;
    return c;
}

template <typename T, int D, int NR>
hipError_t launch(const AttnArgs& a, const AttnShape& shape, hipStream_t s) {
    constexpr int waves = attn_waves(D, 16 * NR);
    constexpr size_t lds = (size_t)waves * 16 * NR * (D + 4 + 2 + kStep) * sizeof(float);
    static LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(k_attn<T, D, NR>), lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attn<T, D, NR>), dim3(shape.grid), dim3(64 * waves), lds, s, a, make_cut(a, shape));
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnShape& shape, hipStream_t s) {
    hipError_t e = hipErrorInvalidValue;
    if (shape.rows == 128)
        e = launch_attn_tile<T, D>(a, make_cut(a, shape), shape, s);
    else if (shape.rows == 16)
        e = launch<T, D, 1>(a, shape, s);
    else if constexpr (D <= 128)
        e = launch<T, D, 2>(a, shape, s);
    if (e != hipSuccess || !shape.bytes) return e;
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

// Items are taken whole or cut.  Cutting costs a launch that waits for the
// first one (measured 5 to 7 us) and the parts' way to memory and back; taking items
// whole costs what the longest of them takes alone.  Both are estimated from the
// longest context and the most new tokens of a sequence, as far as the caller
// knows them.  Measured, a workgroup takes 3 us for a step of k_attn's waves (8 x
// 32 keys of 128: a CU's loads in flight bound it) and 1.5 us for a tile of k_attn_tile.
AttnShape attn_shape(const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int window, int max_query, int max_context) {
    AttnShape s = {};
    const int64_t group = q_heads / c.kv_heads, capacity = (int64_t)b.table_pages * c.page_size.d;
    const int64_t longest = max_query > 0 ? std::min<int64_t>(max_query, tokens) : tokens;  // new tokens of a sequence
    const int64_t most = longest * group;
    const int64_t seqs = std::min<int64_t>(b.seqs, tokens);
    const int cus = compute_units();
    int64_t keys = max_context > 0 ? std::min<int64_t>(max_context, capacity) : capacity;
    if (window) keys = std::min<int64_t>(keys, window + longest);
    double us;  // of a whole item
    int slots;  // workgroups that run at a time
    if (most <= (c.head_dim > 128 ? 16 : 32)) {
        s.rows = most <= 16 ? 16 : 32;
        s.step = kStep;
        slots = cus;
        us = 3.0 * keys * c.head_dim / (256 * 128);
    } else {
        s.rows = 128;
        s.step = 64;
        slots = c.head_dim <= 128 ? 2 * cus : cus;
        us = 1.5 * (keys + 63) / 64 * c.head_dim / 128;
    }
    s.unit = 64;
    s.most_rows = (int)std::min<int64_t>(s.rows, most);
    // Whole: the longest item, or all of them (a sequence's rows see its context
    // less half of the new tokens on average) and half an item for what the last
    // ones run alone.  Cut: ranges of equal units, of which an item counts as
    // many as its sequence's longest.
    const double items = (double)c.kv_heads * (seqs == 1 ? (tokens * group + s.rows - 1) / s.rows : (tokens * group + s.rows * seqs / 2) / s.rows);
    const double mean = window ? us : us * (1.0 - 0.5 * longest / std::max<double>(keys, longest));
    const double parts = std::min<double>(slots, items * keys / s.unit);
    const double join = 7.5 + parts * s.most_rows * c.head_dim * 8 / 4e6;  // written and read at about 4 TB/s
    const double cut = us * items / slots + join;
    const bool whole = items > slots ? mean * items / slots + 0.5 * us <= cut : us <= cut;
    const int64_t bound = item_bound(c, b, q_heads, tokens, s.rows);
    if (whole && bound < (int64_t(1) << 31)) {
        s.unit = 1 << 30;
        s.grid = (int)bound;
        return s;
    }
    // Larger units where this many would pass 31 bits.
    while (s.unit < (1 << 30) && bound * (capacity / s.unit + 1) >= (int64_t(1) << 31)) s.unit *= 2;
    s.grid = slots;
    s.few = items * 8 <= slots;
    s.bytes = (size_t)2 * s.grid * s.rows * (c.head_dim * sizeof(float) + sizeof(f2));
    return s;
}

hipError_t launch_attention(const AttnArgs& a, const AttnShape& shape, int type, hipStream_t s) {
    return type == Q4_TYPE_F16 ? launch_type<F16>(a, shape, s) : launch_type<BF16>(a, shape, s);
}

}  // namespace q4

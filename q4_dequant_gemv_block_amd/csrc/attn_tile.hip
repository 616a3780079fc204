// Attention of many new tokens a sequence (prompts and chunks of them) over a
// paged cache: the same items, units and ranges as k_attn, in tiles that the
// matrix cores are the bound of.
//
// A workgroup of 4 waves holds 64 U query rows and goes through its keys 64 at a
// time.  With U = 2 a wave has 32 rows and all keys; with U = 1, for calls whose rows
// leave the machine idle, two waves share 32 rows, 32 keys of a tile each, and join
// at the end (a prompt of 256 tokens and 40 heads 14.1 -> 11.7 us).  Two workgroups
// share a CU (8 waves of 256 rows that share the tiles were no faster: 606 us
// against 578 for a prompt of 8192).  K and V go from HBM or L2 straight into LDS
// (global_load_lds, 16 bytes a lane), two tiles of each deep, one barrier a tile.
// (A tile begins with the loads of the next V and of the K behind it, then looks up
// the pages of a later tile, and the compiler waits for that lookup at once; loads
// return in order, so the tile's work starts when all of these have landed.  The
// compiler's waits for the queries, in every other tile, come behind that.)
// The products run on v_mfma_f32_32x32x16:
//   S^T = K Q^T: A = 32 keys from LDS, B = Q^T, which stays in registers;
//   O^T = V^T P^T: A = V^T by the transposing LDS read (ds_read_b64_tr_b16: 16
//     lanes read 4 keys of 16 elements and get one element's 4 keys each), B =
//     P^T, which is what the accumulators of S^T hold: lane (h, n) has the keys
//     8 (i / 4) + 4 h + i % 4 of query row n, so the two transposing reads of a 16-key
//     step take keys 4 h .. and 8 + 4 h .. .
// LDS rows are as long as a head; the 16-byte chunk c of row r lies at c ^ f(r),
// so that the 16 rows of a K read and the 4 rows x 64 bytes of a V read cover all 64
// banks (f by row for K, by row % 4 in 64-byte blocks for V; measured without
// conflicts).  The weights' reference is raised as in k_attn.  A wave works on two
// tiles at once: the products of the next tile's scores are issued between the
// exponentials of this one's, so that neither unit waits for the other.
//
// Bound by the matrix cores' issue beside the exponentials.  Measured, heads of 128:
// 2048 tokens over 16384 keys 482 to 514 us (1,002 to 1,069 TFLOP/s with the card's
// clock and the cache; a large library product reaches 1,087 to 1,145), a prompt of
// 8192 551 to 573 (960 to 998), one of 169 tokens 9.1 (latency).
#include "attn_device.h"
#include "q4gemv.h"

namespace q4 {

namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Mma32;
template <>
struct Mma32<F16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f16v mma(u4 a, u4 b, f16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};
template <>
struct Mma32<BF16> {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ f16v mma(u4 a, u4 b, f16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8, a), __builtin_bit_cast(v8, b), c, 0, 0, 0);
    }
};

constexpr int kTile = 64;  // keys of a tile
constexpr int kWaves = 4, kThreads = 64 * kWaves;

// Places in LDS (rows and their swizzles as described above).
template <int D>
struct Layout : LdsRow<D> {
    typedef LdsRow<D> R;
    static constexpr int bytes = kTile * R::row;  // of a tile of K or V
    static __device__ __forceinline__ int swz_v(int r) { return R::chunks == 8 ? ((r >> 1) & 1) << 2 : (r & 3) << 2; }
};

template <typename T, int D, int U, typename WORK>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 2 : 1) k_attn_tile(const AttnArgs a, const Cut cut) {
    typedef Layout<D> L;
    constexpr int NW = kWaves, ROWS = 64 * U;
    constexpr int PAIRS = 8 * U;                       // pairs of scores of a tile a lane has
    constexpr int KS = D / 16;                         // k-steps of the first product
    constexpr int DT = D / 32;                         // 32-element tiles of the output
    constexpr int kAheadK = U * D == 256 ? 3 : 4, kAheadV = U * D == 256 ? 2 : 3;  // LDS reads ahead of the products, as registers allow
    constexpr int LOADS = kTile / L::per_load / NW;    // loads of a wave for K, and for V, of a tile
    constexpr int GROUPS = 8 / NW;                     // groups of 8 keys they cover
    constexpr int PER_GROUP = LOADS / GROUPS;
    extern __shared__ char sh[];  // K [2][64][row], V [2][64][row], then a flag of each wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int h = lane >> 5, n = lane & 31;
    const int rows32 = U == 2 ? wave : wave & 1;      // the wave's 32 rows of the item's
    const int first = U == 2 ? 0 : 32 * (wave >> 1);  // its first key of a tile
    const uint32_t sh0 = lds_address(sh);

    WORK work;
    Item it;
    if (!work.start(cut, a.batch, &it)) return;
    const Seq& seq = work.seq;
    const Parts<D> parts(a.workspace, (int)gridDim.x, ROWS);

    // where this lane reads in a tile: chunks 2 s + h of K's rows, 64-byte block d of V's
    int at_k0 = (first + n) * L::row + ((h ^ L::swz_k(n)) * 16), at_v0;
    {
        const int g = lane >> 4, r = 4 * (g >> 1) + ((lane >> 2) & 3);
        const int c = 2 * (g & 1) + ((lane & 3) >> 1);
        at_v0 = (first + r) * L::row + ((c ^ L::swz_v(r)) * 16) + (lane & 1) * 8;
    }

    while (work.next(cut, a.batch, &it)) {
        const int32_t* table = a.batch.table + seq.b * a.batch.table_stride;
        const char* kbase = a.cache.k + (int64_t)it.head * a.cache.k_head * 2;
        const char* vbase = a.cache.v + (int64_t)it.head * a.cache.v_head * 2;

        // this lane's query row and the wave's first and last positions
        const int row = it.row0 + 32 * rows32 + n;
        const int rc = min(row, it.row0 + it.rows - 1);
        const int qi = (int)cut.group.div(rc), qh = it.head * a.group + rc - qi * a.group;
        const int pos = it.past + qi;
        const int w_rows = min(32, it.rows - 32 * rows32);  // may be <= 0
        const int w_first = it.past + (int)cut.group.div(it.row0 + 32 * rows32);
        const int w_last = it.past + (int)cut.group.div(it.row0 + 32 * rows32 + max(w_rows, 1) - 1);
        u4 qf[KS];
        {
            const char* src = a.q.data + ((int64_t)(seq.row0 + qi) * a.q.token_stride + (int64_t)qh * a.q.head_stride + 8 * h) * 2;
#pragma unroll
            for (int s = 0; s < KS; ++s) qf[s] = *reinterpret_cast<const u4*>(src + 32 * s);
        }
        f16v acc[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
        float m = kNone, l = 0.0f;

        // page of this lane's group (lane % 8) of the tile at key t
        auto pages = [&](int t) { return page_of(a.cache, a.batch, table, t + 8 * (lane & 7)); };
        // K (or V) of the tile at key t into one of its two places
        auto fill = [&](int t, int page8, const char* base, int64_t page_stride, int64_t slot_stride, uint32_t to, bool values) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int group = wave * GROUPS + g;
                const int page = max(__builtin_amdgcn_readlane(page8, group), 0);
                const uint32_t p = (uint32_t)(t + 8 * group);
                const uint32_t slot = p - a.cache.page_size.div(p) * a.cache.page_size.d;
                const char* src = base + ((int64_t)page * page_stride + (int64_t)slot * slot_stride) * 2;
#pragma unroll
                for (int x = 0; x < PER_GROUP; ++x) {
                    const int r8 = x * L::per_load + lane / L::chunks;  // row of the group
                    const int r = 8 * group + r8;
                    const int c = (lane % L::chunks) ^ (values ? L::swz_v(r) : L::swz_k(r));
                    // (heads of 96: the lanes behind a row's end load its last chunks again, for no use: masks for them would cost scalar registers)
                    const int at = D == 8 * L::chunks || c < D / 8 ? c : c - (L::chunks - D / 8);
                    load_to_lds(src, r8 * (uint32_t)slot_stride * 2 + 16 * at, to + (8 * group + x * L::per_load) * L::row);
                }
            }
        };
        auto fill_k = [&](int t, int page8, int stage) {
            fill(t, page8, kbase, a.cache.k_page, a.cache.k_slot, sh0 + stage * L::bytes, false);
        };
        auto fill_v = [&](int t, int page8, int stage) {
            fill(t, page8, vbase, a.cache.v_page, a.cache.v_slot, sh0 + (2 + stage) * L::bytes, true);
        };
        // K fragments (k-step, 32-key half) in the order the products take them
        u4 kf[kAheadK];
        int at_k = at_k0, at_v = at_v0;  // in the tile to read next: toggled, its places are a power of 2 apart
        auto read_k = [&](int i) {
            kf[i % kAheadK] = *reinterpret_cast<const u4*>(sh + (at_k ^ (32 * (i / U))) + i % U * 32 * L::row);
        };
        // V fragments (16 keys, 32 elements)
        u4 vf[kAheadV];
        auto read_v = [&](int i) {
            const char* src = sh + 2 * L::bytes + (at_v ^ (64 * (i % DT))) + 16 * (i / DT) * L::row;
            vf[i % kAheadV] = read_transposed(src, src + 8 * L::row);
        };
        int page0 = 0, page1 = 0, page2 = 0;  // pages of this tile, the next one and the one behind that
        float top;                            // the maximum of the scores in `now` (no masks)

        // S^T of a tile by itself.
        auto scores = [&](f16v (&s)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < U * KS; ++i) {
                read_k(i);
                s[i % U] = Mma32<T>::mma(kf[i % kAheadK], qf[i / U], s[i % U]);
            }
            top = s[0][0];
#pragma unroll
            for (int i = 0; i < 16 * U; ++i) top = fmaxf(top, s[i >> 4][i & 15]);
        };
        f16v even[U], odds[U];  // scores of this tile and of the next one, in turn

        if (it.k_lo < it.k_hi) {
            const int t = it.k_lo;
            page0 = pages(t);
            page1 = pages(t + kTile);
            page2 = pages(t + 2 * kTile);
            __builtin_amdgcn_s_waitcnt(0x0F70);  // with the queries
            fill_k(t, page0, 0);
            fill_v(t, page0, 0);
            if (t + kTile < it.k_hi) {
                fill_k(t + kTile, page1, 1);
                fill_v(t + kTile, page1, 1);
                asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(3 * LOADS) : "memory");  // the first tile's K is there
            } else {
                asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LOADS) : "memory");
            }
            scores(even);
        }
        // One tile: its scores are in `now`, the next one's will be in `next`.
        int stage = 0;
        auto tile = [&](int t, f16v (&now)[U], f16v (&next)[U]) {
            at_k ^= L::bytes;
            asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");  // V of this tile and K of the next are there, the places of K of this one and V of the last free
            const bool more = t + kTile < it.k_hi;
            const int page8 = page0;
            if (more && t > it.k_lo) fill_v(t + kTile, page1, stage ^ 1);  // the second tile's is on its way
            if (t + 2 * kTile < it.k_hi) fill_k(t + 2 * kTile, page2, stage);
            page0 = page1;
            page1 = page2;
            page2 = pages(t + 3 * kTile);
            const uint32_t valid = (uint32_t)__ballot(page8 >= 0) & 0xFF;  // groups with a place

            // Tiles that not all of the workgroup's rows see whole: values of
            // keys that do not belong here become 0, and so do NaN and
            // infinities, which are added below row by row.
            bool odd = false;
            if (valid != 0xFF || t + kTile > min(it.k_hi, it.p_first + 1) || (a.window && t <= it.p_last - a.window)) {
                char* tv = sh + (2 + stage) * L::bytes;
                int thread = threadIdx.x;
                asm volatile("" : "+v"(thread));  // made anew: addresses from it would be held through the loop
                constexpr int MINE = kTile * L::chunks / kThreads;  // chunks a thread looks at
                const bool full = t + kTile <= it.k_hi && valid == 0xFF;
                us2 most = {0, 0};  // the largest magnitude, as bits
#pragma unroll
                for (int k = 0; k < MINE; ++k) {
                    const int u = thread + k * kThreads, r = u / L::chunks;
                    if (D != 8 * L::chunks && ((u % L::chunks) ^ L::swz_v(r)) >= D / 8) continue;
                    u4* at = reinterpret_cast<u4*>(tv + u * 16);
                    if (!full && (t + r >= it.k_hi || !((valid >> (r >> 3)) & 1))) {
                        *at = u4{0, 0, 0, 0};
                        continue;
                    }
                    const u4 v = *at & 0x7FFF7FFFu;
#pragma unroll
                    for (int e = 0; e < 4; ++e) most = __builtin_elementwise_max(most, __builtin_bit_cast(us2, (uint32_t)v[e]));
                }
                constexpr unsigned short infinity = std::is_same<T, F16>::value ? 0x7C00 : 0x7F80;
                const bool mine = max(most.x, most.y) >= infinity;
                if (mine) {
                    for (int u = thread; u < kTile * L::chunks; u += kThreads) {
                        u4* at = reinterpret_cast<u4*>(tv + u * 16);
                        const u4 v = *at;
                        *at = v & ~u4{nonfinite<T>(v.x), nonfinite<T>(v.y), nonfinite<T>(v.z), nonfinite<T>(v.w)};
                    }
                }
                int* flags = reinterpret_cast<int*>(sh + 4 * L::bytes);
                const bool wave_odd = __ballot(mine) != 0;
                if (lane == 0) flags[wave] = wave_odd;
                asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // LDS alone: the next tiles stay in flight
#pragma unroll
                for (int w = 0; w < NW; ++w) odd |= flags[w] != 0;
            }
#pragma unroll
            for (int i = 0; i < kAheadK; ++i) read_k(i);
            if (valid != 0xFF || t + kTile > min(it.k_hi, w_first + 1) || (a.window && t <= w_last - a.window)) {
                uint64_t seen = bits_between(a.window ? pos - a.window + 1 - t : 0, min(it.k_hi, pos + 1) - t);
                if (valid != 0xFF) {  // each group's bit as a byte
                    uint64_t x = valid;
                    x = (x | (x << 28)) & 0x0000000F0000000Full;
                    x = (x | (x << 14)) & 0x0003000300030003ull;
                    x = (x | (x << 7)) & 0x0101010101010101ull;
                    seen &= x * 0xFF;
                }
                seen >>= first + 4 * h;  // the lane's keys are 8 (i / 4) + i % 4 of what is left
                top = kNone;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        now[u][i] = keep_seen(now[u][i], bit_mask((uint32_t)(seen >> (32 * u)), 8 * (i >> 2) + (i & 3)));
                        top = fmaxf(top, now[u][i]);
                    }
            }
            top *= a.scale_log2;
            if (__ballot(top > m + kRaise<T>)) {
                top = fmaxf(top, __shfl_xor(top, 32));
                const float raised = top > m + kRaise<T> ? top - kLift<T> : m;  // each row by itself
                const float f = raised == kNone ? 1.0f : __builtin_amdgcn_exp2f(m - raised);
                m = raised;
                l *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d) acc[d] *= f;
            }
            const float ref = m == kNone ? 0.0f : m;

            // The next tile's scores on the matrix cores while this one's
            // weights are made: a product, a read ahead and a share of the
            // exponentials at a time, those in three stages (exponent, exp2,
            // rounding and sum) so that no instruction waits for the one before.
            u4 p[2 * U];
            constexpr int STEPS = U * KS;
            auto exponent = [&](int j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    now[j >> 3][2 * (j & 7) + e] = __builtin_fmaf(now[j >> 3][2 * (j & 7) + e], a.scale_log2, -ref);
                }
            };
            auto power = [&](int j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    now[j >> 3][2 * (j & 7) + e] = __builtin_amdgcn_exp2f(now[j >> 3][2 * (j & 7) + e]);
                }
            };
            auto weight = [&](int j) {
                p[j >> 2][j & 3] = pack2<T>(now[j >> 3][2 * (j & 7)], now[j >> 3][2 * (j & 7) + 1]);
                l = add_pair<T>(p[j >> 2][j & 3], l);
            };
            // pairs [PAIRS s / STEPS, PAIRS (s + 1) / STEPS) (rounded up) belong to step s
            auto share = [&](int s, auto what) {
#pragma unroll
                for (int e = 0; e < (PAIRS + STEPS - 1) / STEPS; ++e) {
                    const int j = (PAIRS * s + STEPS - 1) / STEPS + e;
                    if (j < (PAIRS * (s + 1) + STEPS - 1) / STEPS && j < PAIRS) what(j);
                }
            };
            share(0, exponent);
            share(1, exponent);
            share(0, power);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) next[u][i] = 0.0f;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                next[s % U] = Mma32<T>::mma(kf[s % kAheadK], qf[s / U], next[s % U]);
                if (s + kAheadK < STEPS) read_k(s + kAheadK);
                if (s >= STEPS - kAheadV) read_v(s - (STEPS - kAheadV));
                share(s + 2, exponent);
                share(s + 1, power);
                share(s, weight);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (odd) {
                // The elements that left the product, for the rows that see them.
                for (int k = first; k < first + 32 * U && t + k < it.k_hi; ++k) {
                    if (!((valid >> (k >> 3)) & 1)) continue;
                    uint32_t w = 0;
#pragma unroll
                    for (int k4 = 0; k4 < 2 * U; ++k4)
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // keys 16 k4 + 8 (j / 2) + 4 h + 2 (j % 2), + 1
                            if (((k - first) & ~5) == 16 * k4 + 8 * (j >> 1) + 2 * (j & 1)) w = p[k4][j];
                    const float weight = half_of<T>((uint32_t)__shfl((int)w, n + 32 * ((k >> 2) & 1)), k & 1);
                    const bool sees = t + k <= pos && (!a.window || t + k > pos - a.window);
                    const int page = __builtin_amdgcn_readlane(page8, k >> 3);
                    const uint32_t slot = (uint32_t)(t + k) - a.cache.page_size.div(t + k) * a.cache.page_size.d;
                    const char* src = vbase + ((int64_t)page * a.cache.v_page + (int64_t)slot * a.cache.v_slot + 4 * h) * 2;
#pragma unroll
                    for (int d = 0; d < DT; ++d)
#pragma unroll
                        for (int i4 = 0; i4 < 4; ++i4) {
                            float v[4];
                            load_elems<T, 4>(src + (32 * d + 8 * i4) * 2, v);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (sees && !__builtin_isfinite(v[i])) acc[d][4 * i4 + i] += weight * v[i];
                            __builtin_amdgcn_sched_barrier(0);  // registers: one load at a time
                        }
                }
            }
            // O^T += V^T P^T, and the maximum of the next tile's scores
            __builtin_amdgcn_s_setprio(1);  // the wave that has its weights goes first: the CU's other waves then have theirs to make (2 to 3 %)
            top = next[0][0];
#pragma unroll
            for (int i = 0; i < 2 * U * DT; ++i) {
                acc[i % DT] = Mma32<T>::mma(vf[i % kAheadV], p[i / DT], acc[i % DT]);
                if (i + kAheadV < 2 * U * DT) read_v(i + kAheadV);
#pragma unroll
                for (int e = 0; e < (8 + DT - 1) / DT; ++e) {
                    const int j = (8 * i + DT - 1) / DT + e;
                    if (j < (8 * (i + 1) + DT - 1) / DT) top = fmaxf(top, next[j >> 4][j & 15]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_s_setprio(0);
            stage ^= 1;
            at_v ^= L::bytes;
        };
        for (int t = it.k_lo; t < it.k_hi; t += 2 * kTile) {
            tile(t, even, odds);
            if (t + kTile < it.k_hi) tile(t + kTile, odds, even);
        }
        __syncthreads();  // all tiles are read before the next item's

        if constexpr (U == 1) {
            // the other 32 keys of each tile, from the wave that has them
            int lane = threadIdx.x & 63;
            asm volatile("" : "+v"(lane));
            f4* other = reinterpret_cast<f4*>(sh) + (rows32 * DT * 4) * 64 + lane;
            f2* other_ml = reinterpret_cast<f2*>(sh + 2 * DT * 4 * 64 * sizeof(f4)) + rows32 * 64 + lane;
            if (first) {
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        other[(4 * d + i) * 64] = f4{acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
                *other_ml = f2{m, l};
            }
            __syncthreads();
            if (!first) {
                const f2 ml = *other_ml;
                const float both = fmaxf(m, ml.x), ref = both == kNone ? 0.0f : both;
                const float f0 = __builtin_amdgcn_exp2f(m - ref), f1 = __builtin_amdgcn_exp2f(ml.x - ref);
                m = both;
                l = l * f0 + ml.y * f1;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f4 o = other[(4 * d + i) * 64];
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[d][4 * i + e] = acc[d][4 * i + e] * f0 + o[e] * f1;
                    }
            }
            __syncthreads();
            if (first) {
                if constexpr (WORK::once) break;
                continue;
            }
        }
        l += __shfl_xor(l, 32);
        // (lane numbers anew: addresses made from them would be held through the loop)
        int n = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
        asm volatile("" : "+v"(n), "+v"(h));
        if (32 * rows32 + n >= it.rows) {
            if constexpr (WORK::once) break;
            continue;
        }
        if (work.whole(it)) {
            const float f = row_scale(l);
            char* dst = a.out.data + ((int64_t)(seq.row0 + qi) * a.out.token_stride + (int64_t)qh * a.out.head_stride + 4 * h) * 2;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float v[4] = {acc[d][i] * f, acc[d][i + 1] * f, acc[d][i + 2] * f, acc[d][i + 3] * f};
                    store_elems<T, 4>(dst + (32 * d + 2 * i) * 2, v);
                }
            if (a.lse && h == 0) a.lse[(int64_t)(seq.row0 + qi) * a.q_heads + qh] = row_lse(m, l);
        } else {
            const int64_t slot = ((int64_t)2 * blockIdx.x + (it.u0 == 0)) * ROWS + 32 * rows32 + n;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<f4*>(&parts.o[slot * D + 32 * d + 2 * i + 4 * h]) = f4{acc[d][i], acc[d][i + 1], acc[d][i + 2], acc[d][i + 3]};
            if (h == 0) parts.ml[slot] = f2{m, l};
        }
        if constexpr (WORK::once) break;
    }
}

template <typename T, int D, int U, typename WORK>
hipError_t launch_work(const AttnArgs& a, const Cut& cut, const AttnShape& shape, hipStream_t s) {
    constexpr size_t lds = (size_t)4 * Layout<D>::bytes + kWaves * sizeof(int);
    static LdsLimit limit;
    const hipError_t e = limit.raise(reinterpret_cast<const void*>(k_attn_tile<T, D, U, WORK>), lds);
    if (e != hipSuccess) return e;
    return launch_shape(shape, cut, [&](unsigned grid, const Cut& c) {
        hipLaunchKernelGGL((k_attn_tile<T, D, U, WORK>), dim3(grid), dim3(kThreads), lds, s, a, c);
    });
}

template <typename T, int D, int U>
hipError_t launch(const AttnArgs& a, const Cut& cut, const AttnShape& shape, hipStream_t s) {
    return shape.places ? launch_work<T, D, U, Places>(a, cut, shape, s) : launch_work<T, D, U, Work>(a, cut, shape, s);
}

}  // namespace

template <typename T, int D>
hipError_t launch_attn_tile(const AttnArgs& a, const Cut& cut, const AttnShape& shape, hipStream_t s) {
    return shape.rows == 128 ? launch<T, D, 2>(a, cut, shape, s) : launch<T, D, 1>(a, cut, shape, s);
}

template hipError_t launch_attn_tile<F16, 64>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<F16, 96>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<F16, 128>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<F16, 256>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 64>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 96>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 128>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 256>(const AttnArgs&, const Cut&, const AttnShape&, hipStream_t);

}  // namespace q4

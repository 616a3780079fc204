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
#include "attn_rows.h"
#include "attn_shape.h"

#include <atomic>

namespace q4 {

namespace {

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

AttnShape attn_shape(const CacheArg& c, const BatchArg& b, int q_heads, int64_t tokens, int window, int max_query, int max_context, bool tree) {
    return attn_shape_on(compute_units(), c, b, q_heads, tokens, window, max_query, max_context, tree);
}

size_t attn_most_bytes(int head_dim, int64_t rows) { return attn_workspace_most(compute_units(), head_dim, rows); }

hipError_t launch_attention(const AttnArgs& a, const AttnShape& shape, int type, hipStream_t s) {
    return type == Q4_TYPE_F16 ? launch_type<F16>(a, shape, s) : launch_type<BF16>(a, shape, s);
}

}  // namespace q4

// Attention of trees of drafted tokens over a paged key/value cache (gfx950).
//
// Each new token sees the tokens that are in the cache and, of its own sequence's new
// ones, those that its mask names (its ancestors and itself): the items, units, loads
// and products of the causal kernels (attn_rows.h, attn_tile.h), with other masks in
// the steps that reach new tokens.  A row's mask is a string of bits by token; the 32
// or 64 bits of a step's keys are cut out of it by two shifts, and what lies in front
// of the new tokens is seen whole, or, with a window, from past + depth - window + 1 on
// (depth: the new tokens that the row sees beside itself).  Steps in front of the new
// tokens pay nothing.
//
// A tree's rows are few and its keys many, so the tiles' waits count: here the pages of
// 32 tiles are looked up at once into LDS, so that a tile waits for no load but its own
// (whole items of 64 rows over 4000 keys 106 -> 74 us), the parts are joined by item, a
// row a group of lanes (34 -> 11 us for 3 sequences of 64 tokens), and waves without
// rows do their loads alone.
//
// Items of 256 rows (trees of more than 128 rows of a kv head, heads of 96 and 128) are
// taken by two workgroups, half of the rows each, that run at once on one XCD: the keys
// come from HBM once and to the second one from the L2, and a CU's two workgroups hide
// each other's waits (a workgroup of 8 waves that share the tiles in LDS took 6 % longer,
// items of 128 rows by themselves 16 %, over 3 sequences of 64 tokens over 32768 keys).
//
// Measured, 32 query heads over 8 of 128, a call: 16 ragged sequences of up to 33 tokens
// over up to 6001 keys 74 us (3.1 TB/s of keys and values; the matrix products of rows
// that are there take 20, HBM 32 at 7.2 TB/s; a workgroup has about 1.5 items of 27
// tiles, whose start and end, some 8 us, nothing hides), 3 of 64 over 32768 keys 140
// (738 TFLOP/s; 792 in the kernel; 88 us at the rate of a large product), one of 16 tokens
// over 515 keys of 40 heads 10.1 (latency).
// Tried: four tiles of K and of V in LDS for 8 waves instead of two (71 and 141 us, as
// before: not the loads are what is waited for); weights summed a step after they are
// packed (no change).
#include "attn_rows.h"

namespace q4 {

namespace {

template <typename T>
hipError_t launch_type(const TreeArgs& a, const AttnShape& shape, hipStream_t s) {
    switch (a.cache.head_dim) {
        case 64: return launch_dim<T, 64>(a, shape, s);
        case 96: return launch_dim<T, 96>(a, shape, s);
        case 128: return launch_dim<T, 128>(a, shape, s);
        default: return launch_dim<T, 256>(a, shape, s);
    }
}

}  // namespace

hipError_t launch_attention_tree(const TreeArgs& a, const AttnShape& shape, int type, hipStream_t s) {
    return type == Q4_TYPE_F16 ? launch_type<F16>(a, shape, s) : launch_type<BF16>(a, shape, s);
}

}  // namespace q4

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

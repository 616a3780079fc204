// Attention of wide trees of drafted tokens: the tiles of attn_tile.h with the masks
// of attn_tree.hip.
#include "attn_tile.h"

namespace q4 {

template <typename T, int D>
hipError_t launch_attn_tile(const TreeArgs& a, const Cut& cut, const AttnShape& shape, hipStream_t s) {
    if constexpr (D == 96 || D == 128)
        if (shape.rows == 256) return launch_work<T, D, 2, WorkOf<true, true>>(a, cut, shape, s);  // (never taken whole)
    return shape.rows == 128 ? launch<T, D, 2>(a, cut, shape, s) : launch<T, D, 1>(a, cut, shape, s);
}

template hipError_t launch_attn_tile<F16, 64>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<F16, 96>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<F16, 128>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<F16, 256>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 64>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 96>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 128>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);
template hipError_t launch_attn_tile<BF16, 256>(const TreeArgs&, const Cut&, const AttnShape&, hipStream_t);

}  // namespace q4

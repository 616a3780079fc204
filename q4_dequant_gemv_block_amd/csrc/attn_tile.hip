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
#include "attn_tile.h"

namespace q4 {

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

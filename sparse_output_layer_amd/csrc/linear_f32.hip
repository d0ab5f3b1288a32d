// linear_f32.hip -- the fp32 instances of the tiled product (linear_tile.h)
// and the choice of the tile: the matrix cores' fp32 rate is a sixteenth of
// their bf16 rate, so that tiles of 128 x 128 are far from the LDS's bound.
#include "linear_tile.h"

namespace haste {

template <bool PK, bool QK, int ACT>
static hipError_t pick(const LinArgs &a, hipStream_t st) {
    auto tiles = [&](int64_t tl, int64_t tb) { return ((a.N + tl - 1) / tl) * ((a.M + tb - 1) / tb) * a.splits; };
    auto grid = [&](int64_t T, int wg_per_cu) {
        const int64_t up = (T + 7) / 8 * 8, most = 256 * wg_per_cu;
        return dim3((unsigned)(up < most ? up : most));
    };
    const int64_t mid = tiles(128, 128), few = tiles(64, 64);
    if (few > INT32_MAX - 8) return hipErrorInvalidValue;
    // 1024 -> 1024, rows and us of the tiles 128, 64: 1024 72, 29; 2048 74, 46; 4096
    // 79, 78; 8192 139, 147.  Partial products (splits) are made for 64 x 64.
    if (a.splits == 1 && mid >= 192) hipLaunchKernelGGL((k_linear_tile<false, PK, QK, 2, 2, false, ACT>), grid(mid, 2), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_linear_tile<false, PK, QK, 1, 4, false, ACT>), grid(few, 4), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_linear_f32(const LinArgs &a, bool pk, bool qk, int act, hipStream_t st) {
    if (pk && qk) {
        switch (act) {
        case 0: return pick<true, true, 0>(a, st);
        case 1: return pick<true, true, 1>(a, st);
        case 2: return pick<true, true, 2>(a, st);
        default: return pick<true, true, 3>(a, st);
        }
    }
    return pk ? pick<true, false, 0>(a, st) : pick<false, false, 0>(a, st);
}

}  // namespace haste

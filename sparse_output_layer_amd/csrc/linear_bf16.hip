// linear_bf16.hip -- the bf16 instances of the tiled product (linear_tile.h)
// and the choice of the tile.
#include "linear_tile.h"

namespace haste {

template <bool PK, bool QK, bool YB, int ACT>
static hipError_t pick(const LinArgs &a, hipStream_t st) {
    auto tiles = [&](int64_t tl, int64_t tb) { return ((a.N + tl - 1) / tl) * ((a.M + tb - 1) / tb) * a.splits; };
    auto grid = [&](int64_t T, int wg_per_cu) {
        const int64_t up = (T + 7) / 8 * 8, most = 256 * wg_per_cu;
        return dim3((unsigned)(up < most ? up : most));
    };
    const int64_t big = tiles(256, 256), mid = tiles(128, 128), few = tiles(64, 64);
    if (few > INT32_MAX - 8) return hipErrorInvalidValue;
    // 1024 -> 1024, rows and us of the tiles 256, 128, 64: 2048 25, 12.1, 11.1; 4096
    // 27, 13.9, 17.6; 8192 29, 22.5, 30; 12288 31, 32.5, 43; 16384 36, 42, 63 (of 144
    // tiles of 128 x 128, a weight gradient's: 20.8, in 64 x 64 23.1)
    if (big >= 192) hipLaunchKernelGGL((k_linear_tile<true, PK, QK, 4, 1, YB, ACT>), grid(big, 1), dim3(256), 0, st, a);
    else if (mid >= 144) hipLaunchKernelGGL((k_linear_tile<true, PK, QK, 2, 2, YB, ACT>), grid(mid, 2), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_linear_tile<true, PK, QK, 1, 4, YB, ACT>), grid(few, 4), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_linear_bf16(const LinArgs &a, bool pk, bool qk, bool yb, int act, hipStream_t st) {
    if (pk && qk) {
        switch (act) {
        case 0: return yb ? pick<true, true, true, 0>(a, st) : pick<true, true, false, 0>(a, st);
        case 1: return yb ? pick<true, true, true, 1>(a, st) : pick<true, true, false, 1>(a, st);
        case 2: return yb ? pick<true, true, true, 2>(a, st) : pick<true, true, false, 2>(a, st);
        default: return yb ? pick<true, true, true, 3>(a, st) : pick<true, true, false, 3>(a, st);
        }
    }
    if (pk) return yb ? pick<true, false, true, 0>(a, st) : hipErrorInvalidValue;
    return yb ? pick<false, false, true, 0>(a, st) : pick<false, false, false, 0>(a, st);
}

}  // namespace haste

// linear_plan.hpp -- which kernels a whole linear takes (host).
#pragma once

#include <stdint.h>

#include "internal.hpp"

namespace dmpq {

enum LinearRoute { kLinearBF16, kLinearInt8, kLinearNVFP4 };

// Which kernels a whole linear takes.
// kPathFew reads the weight once over the whole chip, 16 columns a workgroup: up to 16 rows, and more while the product is small (us, few / mid, bf16: 16 x 1920 x
// 1920 6.5 / 9.1, 32 rows 8.2 / 9.1, 64 rows 11.9 / 9.3; 226 x 600 x 688 5.2 / 8.5).
// kPathMid has tiles of 64 and 128, for products whose 256 x 256 tiles leave much
// of the chip idle.  Those take about the same for any number of them up to 256,
// and K long enough to be split shortens it (us, mid / tiles: bf16 900 x 1920 x 1920
// 16 / 39, 900 x 5760 x 1920 43 / 46, 900 x 7680 x 1920 56 / 51, 900 x 1920 x 7680 46 / 52,
// 1700 x 1920 x 7680 93 / 71; INT8 900 x 7680 x 1920 38 / 38, 1700 x 1920 x 7680 52 / 51;
// NVFP4 450 x 7680 x 1920 40 / 42, 900 x 5760 x 1920 57 / 48, 900 x 1920 x 7680 71 / 53).
// The fused amax comes from tiles.
enum LinearPath { kPathFew, kPathMid, kPathTiles };
inline LinearPath linear_path(LinearRoute route, bool amax, int64_t M, int64_t N, int64_t K) {
    // 256 x 256 tiles up to which the middling kernels are taken: K below 4096, and from there on
    constexpr int most[3][2] = {{92, 40}, {120, 56}, {60, 24}};
    const int bytes = route == kLinearInt8 ? 1 : 2;  // of a value as the MFMA takes it (NVFP4: as fp16)
    if (!amax && N <= kMaxFewWidth && M <= kMaxFewRows &&
        (M <= 16 || (M + 15) / 16 * 16 * N <= (int64_t(1) << 28) / (K * bytes)))
        return kPathFew;
    return gemm_tiles(M, N) <= most[route][K >= 4096] ? kPathMid : kPathTiles;
}

// The tiles of a middling product (wide: with heads of 128).  A CU holds one tile at a time, and a round of 256 of them takes about (K = 1920,
// us, BF16 / INT8) 9 / 6 with 64 x 64, 14.5 / 10 with 64 x 128 and 25 / 18 with 128 x 128: the
// smallest as long as it is one round, 128 x 128 where it takes at most 4/7 of the
// rounds of 64 x 128 (1693 x 1920 x 1920: 28.9 / 19.7 and 25.9 / 18.4).  NVFP4: 64 x 64, and 32 x
// 128 for heads of 128, which need a tile of their width.
struct MidTile {
    int rows, cols;
};
inline MidTile mid_tile(LinearRoute route, bool wide, int64_t M, int64_t N) {
    if (route == kLinearNVFP4) return wide ? MidTile{32, 128} : MidTile{64, 64};
    const int64_t m64 = (M + 63) / 64, n64 = (N + 63) / 64, n128 = (N + 127) / 128;
    const int64_t wides = m64 * n128, larges = (M + 127) / 128 * n128;
    if (!wide && (larges + 255) / 256 * 7 <= (wides + 255) / 256 * 4) return MidTile{128, 128};
    return m64 * n64 > 256 || wide ? MidTile{64, 128} : MidTile{64, 64};
}

}  // namespace dmpq

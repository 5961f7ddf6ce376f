// linear_plan.hpp -- which kernels a whole linear takes (host).
#pragma once

#include <stdint.h>

#include "internal.hpp"

namespace dmpq {

enum LinearRoute { kLinearBF16, kLinearInt8, kLinearNVFP4 };

// Which kernels a whole linear takes.
// kPathFew reads the weight once over the whole chip, 16 columns a workgroup: up to
// 16 rows, and more while the product is small (us, few / mid: BF16 16 x 1920 x 1920
// 6.3 / 9.0, 32 rows 8.3 / 9.0, 64 rows 11.8 / 9.6, 16 x 7680 x 1920 10.4 / 9.9, 32 rows 13.9 /
// 10.1, 226 x 608 x 688 5.0 / 7.9; INT8 64 x 1920 x 1920 7.7 / 7.2; NVFP4 11.1 / 10.3).
// kPathMid has tiles of 64 and 128, for products whose 256 x 256 tiles leave much
// of the chip idle.  Those take about the same for any number of them up to 256,
// and K long enough to be split shortens it (us, mid / tiles: BF16 900 x 1920 x 1920
// 16 / 34, 900 x 5760 x 1920 40 / 42, 900 x 7680 x 1920 46 / 55, 2900 x 1920 x 1920 39 / 41,
// 900 x 1920 x 7680 41 / 51, 1700 x 1920 x 7680 66 / 71; INT8 900 x 7680 x 1920 33 / 33,
// 3400 x 1920 x 1920 33 / 34, 1700 x 1920 x 7680 40 / 48; NVFP4 450 x 7680 x 1920 40 / 40,
// 2000 x 1920 x 1920 37 / 39, 900 x 5760 x 1920 55 / 44, 450 x 1920 x 7680 35 / 37, 900 x 1920 x
// 7680 66 / 49).  BF16 900 x 7680 x 1920 and 1700 x 1920 x 7680 are beyond the limits, though
// the middling kernels' 128 x 128 tiles are 15 and 7% faster there.
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

// The tiles of a middling product (wide: with heads of 128).  A CU holds one tile at a
// time, and a full round of 256 of them takes (K = 1920, us, BF16 / INT8) 11.5 / 8.2 with
// 64 x 64, 15.6 / 11.3 with 64 x 128 and 25 / 18.5 with 128 x 128:
// the smallest as long as it is one round, 128 x 128 where it takes at most 4/7 of the
// rounds of 64 x 128 (1693 x 1920 x 1920 BF16 64 x 128 27.6, 128 x 128 24.5; INT8 19.5 and
// 18.0; 1700 x 1920 x 7680 81 and 66, 48 and 40).  NVFP4: 64 x 64, and 32 x 128 for heads of
// 128, which need a tile of their width.
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

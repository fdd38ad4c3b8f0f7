// Sizes and launch geometry of the 8-bit matrices and their products; like zs_grid.h plain
// C++, checked on the host alone.
#pragma once

#include "zs_grid.h"

namespace zs {

constexpr int kF8Block = 128;                      // elements to a scale byte along a row
constexpr int64_t kF8MaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kF8MaxCols = int64_t(1) << 22;   // 256 rows of codes stay under 2^31 bytes

constexpr int64_t f8_ceil(int64_t a, int64_t b) { return a / b + (a % b != 0 ? 1 : 0); }
inline int64_t f8_ld(int64_t cols) { return f8_ceil(cols, kF8Block) * kF8Block; }
inline int64_t f8_lds(int64_t cols) { return f8_ceil(cols, 4 * kF8Block) * 4; }
inline int64_t f8_code_bytes(int64_t rows, int64_t cols) { return rows * f8_ld(cols); }
inline int64_t f8_scale_bytes(int64_t rows, int64_t cols, int block_rows) {
    return f8_ceil(rows, block_rows) * f8_lds(cols);
}

// Quantisation and its inverse: one workgroup per 128 x 128 tile.
inline int64_t f8_tiles(int64_t rows, int64_t cols) {
    return f8_ceil(rows, kF8Block) * f8_ceil(cols, kF8Block);
}
inline int64_t f8_tile_grid(int64_t tiles) { return grid_blocks(tiles, 1); }

// How a product is cut: tiles of tm x tn of C, each summed by `splits` workgroups.
struct F8Plan {
    int tm, tn;
    int splits;
    int64_t tiles_m, tiles_n;
};
// Counts of the workgroups that are done with a tile stand first in the workspace, at the
// same place whatever the sizes (0 between calls): of a call's first product, then of its
// second. A product that is split has fewer tiles than that.
constexpr int64_t kF8Counts = 1024;
constexpr int64_t kF8CountBytes = 2 * kF8Counts * 4;

inline F8Plan f8_plan(int64_t M, int64_t N, int64_t K, bool exact) {
    (void)exact;
    if (f8_ceil(M, 256) * f8_ceil(N, 256) >= 200)
        return F8Plan{256, 256, 1, f8_ceil(M, 256), f8_ceil(N, 256)};
    F8Plan p{128, 128, 1, f8_ceil(M, 128), f8_ceil(N, 128)};
    const int64_t blocks = f8_ceil(K, kF8Block);
    if (p.tiles_m * p.tiles_n < 256) {
        p = F8Plan{64, 64, 1, f8_ceil(M, 64), f8_ceil(N, 64)};
        const int64_t t = p.tiles_m * p.tiles_n;
        if (t > 0 && t < 256) {
            int64_t s = 512 / t;
            if (s > blocks / 4) s = blocks / 4;
            p.splits = int(s < 1 ? 1 : (s > 16 ? 16 : s));
        }
    }
    return p;
}
inline int64_t f8_partial_bytes(const F8Plan& p) {
    return p.splits > 1 ? p.tiles_m * p.tiles_n * p.splits * p.tm * p.tn * 4 : 0;
}
inline int64_t f8_matmul_workspace(int64_t M, int64_t N, int64_t K) {
    const int64_t a = f8_partial_bytes(f8_plan(M, N, K, false)),
                  b = f8_partial_bytes(f8_plan(M, N, K, true));
    const int64_t most = a > b ? a : b;
    return most > 0 ? kF8CountBytes + most : 0;
}

}  // namespace zs

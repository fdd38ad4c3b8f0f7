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

// Quantisation: one workgroup of 512 threads per 128 x 128 tile, as many as keep the launch's
// threads below 2^32 (2^23 - 1). Its inverse: one of 256 threads per 64 x 128.
constexpr int kF8TileThreads = 512;
inline int64_t f8_tiles(int64_t rows, int64_t cols) {
    return f8_ceil(rows, kF8Block) * f8_ceil(cols, kF8Block);
}
inline int64_t f8_quant_grid(int64_t tiles) {
    constexpr int64_t most = ((int64_t(1) << 32) - 1) / kF8TileThreads;
    return tiles < 1 ? 1 : (tiles < most ? tiles : most);
}
inline int64_t f8_values_grid(int64_t rows, int64_t cols) {
    return grid_blocks(f8_ceil(rows, 64) * f8_ceil(cols, kF8Block), 1);
}

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

// Products with few rows of a: workgroups of 8 reading wavefronts with an equal share of b's
// rows each (F8Plan's tn; 4 at least), on every CU one; `splits` of the wavefronts take 16
// rows together. LDS holds one or two groups of b for each wavefront, and all of a.
constexpr int kF8Few = 16, kF8FewWaves = 8;
constexpr int64_t kF8FewSums = 2 * kF8FewWaves * 64 * 16, kF8FewGroup = 16 * 512 + 256;
constexpr int64_t kF8FewLds = 163840;
constexpr int64_t f8_few_lds(int depth, int64_t M, int64_t blocks) {
    return kF8FewWaves * depth * kF8FewGroup + kF8FewSums + M * (blocks * kF8Block + 16 + blocks);
}

// Tiles of 256, 128 or 64 squared: the larger one moves less through LDS for each product,
// the smaller ones fill 256 CUs with less. The costs of a step of 128 along K for each tile
// that a CU takes are measured, in hundredths of a microsecond, for C in bf16. C in fp32 is cut
// alike, since the workspace is asked for by sizes alone; its own costs, 290, 93 and 33, favour
// small tiles more, so that it loses where rounds of tiles fall badly (2624 x 11840 x 4096 by
// 256 293, by 128 241; 3000 x 3000 x 3000 71, 68) and wins as much elsewhere (384 x 10944 x 4096
// 50 by 128, 58 by the 64 in one part that those costs pick). Measured with the same operands
// again, in us, M x N x K and C in bf16: 3000 x 3000 x 3000
// 256: 39, 128: 46, 64: 58; 2048 x 4096 x 4096 47, 43, 67; 512 x 4096 x 4096 46, 19, 17.
// CUs that tiles of 128 or 64 leave idle take parts of K, of 16 steps at least, if joining them
// (writing the partial sums, and one workgroup a tile reading its own again) costs less than
// the steps it saves: 512 x 4096 x 11008 64: 47, 128: 51, 128 in 2 parts: 37; 256 x 256 x 8192
// 64 in 1, 2, 4 parts 19, 13, 10; 1024 x 1024 x 4096 64 in 1 and 2 parts 11, 13. (256 in 2 parts
// would gain where K is past 10,000 alone, 2048 x 4096 x 11008 99 for 114, and take 64 MiB.)
// With other operands in turn, from memory, these products take 5 to 7 us more
// (512 x 4096 x 11008 46 to 48).
inline F8Plan f8_plan(int64_t M, int64_t N, int64_t K) {
    constexpr int kCus = 256;
    const int side[3] = {256, 128, 64}, cost[3] = {150, 58, 25};
    F8Plan best{};
    int64_t least = -1;
    const int64_t blocks = f8_ceil(K, kF8Block);
    if (M <= kF8Few && f8_few_lds(1, M, blocks) <= kF8FewLds) {
        const int64_t rows = f8_ceil(N, kCus);
        int s = 1;
        while (s < kF8FewWaves && s * 8 <= blocks) s *= 2;
        return F8Plan{kF8Few, int(rows < 4 ? 4 : rows), s, 1, f8_ceil(N, rows < 4 ? 4 : rows)};
    }
    for (int i = 0; i < 3; ++i) {
        F8Plan p{side[i], side[i], 1, f8_ceil(M, side[i]), f8_ceil(N, side[i])};
        const int64_t tiles = p.tiles_m * p.tiles_n;
        int64_t c = f8_ceil(tiles, kCus) * cost[i] * (blocks > 0 ? blocks : 1);
        int64_t s = tiles > 0 ? kCus / tiles : 0;
        s = s < blocks / 16 ? s : blocks / 16;
        s = s < 32 ? s : 32;
        if (i > 0 && s > 1) {
            // 2 us, 0.35 us a MB of all partial sums and 10 us a MB of one tile's
            const int64_t kb = s * side[i] * side[i] * 4 / 1000;
            const int64_t joined = cost[i] * f8_ceil(blocks, s) + 200 + tiles * kb * 35 / 1000 + kb;
            if (joined < c) c = joined, p.splits = int(s);
        }
        if (least < 0 || c < least) best = p, least = c;
    }
    return best;
}
// Whether a linear layer's product makes a's codes on the way, in every workgroup those of its
// own rows: one launch instead of two, where a CU takes one tile at most and K is short enough
// that making the same codes again for every 64 columns costs less than a launch. Measured, us,
// one launch against two, bf16, the same operands again: 17 x 64 x 128 3.9, 5.5; 512 x 512 x 256 5.3, 7.1;
// 1000 x 1000 x 512 6.5, 8.3; 2048 x 256 x 1024 8.6, 9.9; 256 x 4096 x 1024 9.1, 9.3;
// 777 x 1001 x 1500 12.6, 12.4; 200 x 300 x 2048 13.5, 11.
constexpr int kF8MadeSide = 64, kF8MadeBlocks = 8;
inline bool f8_made(const F8Plan& p, int64_t K) {
    return p.tm == kF8MadeSide && p.splits == 1 && p.tiles_m * p.tiles_n <= 256 && K > 0 &&
           K <= kF8MadeBlocks * kF8Block;
}
inline int64_t f8_partial_bytes(const F8Plan& p) {
    return p.splits > 1 && p.tm != kF8Few ? p.tiles_m * p.tiles_n * p.splits * p.tm * p.tn * 4 : 0;
}
inline int64_t f8_matmul_workspace(int64_t M, int64_t N, int64_t K) {
    const int64_t n = f8_partial_bytes(f8_plan(M, N, K));
    return n > 0 ? kF8CountBytes + n : 0;
}

}  // namespace zs

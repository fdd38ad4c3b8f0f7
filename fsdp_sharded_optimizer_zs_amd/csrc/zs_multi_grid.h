// Launch geometry of the kernels over many tensors, of the 8-bit moments and of the
// 4-bit shards; like zs_grid.h plain C++, checked on the host alone.
#pragma once

#include "zs_grid.h"

namespace zs {

// Conversions of 8-bit moments: one wavefront per `blocks` blocks of 256 elements.
inline int64_t state8_grid(int64_t S, int blocks) {
    const int64_t per = int64_t(blocks) * 256;
    return grid_blocks(S / per + (S % per != 0), kBlockThreads / 64);
}

// The norm over a table's chunks: workgroups of 16 wavefronts, 4 to a chunk, at most 2 on
// each of 256 CUs (which fills them), whose partial sums fit zs_grad_norm's workspace; one
// if there is nothing.
constexpr int kNormThreads = 1024;
constexpr int64_t kNormChunks = 4;
constexpr int64_t kNormGrid = 512;
inline int64_t norm_grid(int64_t n_chunks) {
    const int64_t b = n_chunks / kNormChunks + (n_chunks % kNormChunks != 0);
    return b < 1 ? 1 : (b < kNormGrid ? b : kNormGrid);
}

// 4-bit quantisation of values of es bytes: one workgroup per tile of kMx4Groups 16-byte
// groups of values a lane.
constexpr int kMx4Groups = 2;
inline int64_t quantize_mx4_grid(int64_t S, int es) {
    const int64_t tile = int64_t(kBlockThreads) * (16 / es) * kMx4Groups;
    return grid_blocks(S / tile + (S % tile != 0), 1);
}

// Gather from 4-bit shards: the same tiles, a row of the grid per shard (the whole grid
// under the cap).
inline int64_t gather_mx4_grid(int64_t S, int es, int D) {
    const int64_t b = quantize_mx4_grid(S, es), cap = kMaxGrid / D;
    return b < cap ? b : cap;
}

}  // namespace zs

// Block-scaled 8-bit matrices for gfx950: quantisation of a bf16 or fp32 matrix (as it is
// and transposed, from one read), the same of a matrix that lies in a unit's shards, and
// the values that codes stand for.
//
// All stream once over their data. A workgroup of 8 wavefronts takes a 128 x 128 tile, so
// that the blocks of both forms are whole in it. Lane l of wavefront w holds 8 columns
// (from 8 (l % 16) on) of the rows 16 w + 4 (l / 16) + i, i < 4: 16 lanes cover 256 bytes of a
// bf16 row, a row's block of 128 is the 16 lanes of a DPP row, and the 4 rows i of a column
// are one word of transposed codes. Those words are exchanged through LDS (16 KiB) so that the
// transpose leaves in 16-byte pieces of whole 128-byte runs too.
//
// Memory bounds them: 2 or 4 bytes read and 1 written for each element and form. Measured with
// 1.2 GB of matrices in turn, so that they come from HBM, launches in a row, 4096 x 11008 in us
// (TB/s), as it is / transposed / both / both from 4 shards:
//   bf16, blocks of 1 x 128      29.4 (4.6) / 29.8 (4.5) / 40.5 (4.5) / 43.4
//   bf16, 128 x 128              28.4 (4.8) / 29.0 (4.7) / 38.2 (4.7) / 38.5
//   fp32, 1 x 128                51.8 (4.4) / 53.3 (4.2) / 61.5 (4.4) / 66.3
//   fp32, 128 x 128              47.5 (4.7) / 50.7 (4.4) / 58.0 (4.7) / 59.7
// and back to bf16 26.4 (5.1). Tiles by 4 wavefronts of twice the rows, with four matrices in turn,
// against these: 28.5, 28.0, 39.5 and 49.0 in the first line for 27.9, 28.5, 37.5 and 43.6, in
// the second 24.5, 25.5, 33.2, 40.0 for 26.6, 27.7, 35.0, 39.4; a small matrix, whose tiles
// leave CUs idle, takes longer by them (2048 x 1024, both forms 6.5 us against 5.6, from shards
// 7.5 against 5.7), and fp32 needs twice the registers.

#include "zs_f8_dev.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = kBlockThreads;
constexpr int kTileThreads = kF8TileThreads, kWaves = kTileThreads / 64;  // of a tile to be quantised
constexpr int kT = kF8Block;  // side of a tile

// A matrix in memory, row r from element r * ldx on.
struct Strided {
    const void* x;
    int64_t ldx;
    template <int DT>
    __device__ __forceinline__ Eight<DT> get(int64_t r, int64_t c, int live) const {
        if (live >= 8) return load8<DT>(x, r * ldx + c);
        Eight<DT> v{};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < live) load1<DT>(x, r * ldx + c + e, e, v);
        return v;
    }
};

// A matrix in a unit's shards: the shard of an element by a product with 1 / S in fp64
// (elements are below 2^53, so that it is off by at most one, which is put right).
struct Sharded {
    const F8Shards* s;
    int64_t cols;
    __device__ __forceinline__ int shard_of(int64_t f, int64_t* at) const {
        int r = int(double(f) * s->inv_s);
        int64_t i = f - int64_t(r) * s->S;
        if (i < 0) --r, i += s->S;
        if (i >= s->S) ++r, i -= s->S;
        *at = i;
        return r;
    }
    template <int DT>
    __device__ __forceinline__ Eight<DT> get(int64_t r, int64_t c, int live) const {
        int64_t i;
        int k = shard_of(s->offset + r * cols + c, &i);
        if (live >= 8 && i + 8 <= s->S) return load8<DT>(s->shards.p[k], i);
        Eight<DT> v{};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < live) load1<DT>(s->shards.p[k], i, e, v);
            // every shard ends at a multiple of S: the next element is the next one's first
            if (++i >= s->S) {
                i = 0;
                if (e + 1 < live) ++k;
            }
        }
        return v;
    }
};

// The scale byte of block `block` of row `row`, and, beside the last one, the bytes 1 that
// fill the row: lane k < 4 writes byte block + k.
__device__ __forceinline__ void put_scale(const F8Out& o, int64_t row, int64_t block,
                                          int64_t blocks, int k, int s) {
    if (k == 0 || (block + 1 == blocks && block + k < o.lds))
        global<g_u8>(o.scales)[row * o.lds + block + k] = uint8_t(k == 0 ? s : 1);
}

struct Shared {
    uint32_t codes[kT * kT / 4];
    uint32_t top[kWaves][kT];
    __attribute__((aligned(16))) int scale[kT];
    uint32_t whole[kWaves];
};
__device__ __forceinline__ uint32_t max_of(const uint32_t* x, int step) {
    uint32_t u = x[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) u = max_u(u, x[w * step]);
    return u;
}

// A lane's elements of a tile, rows 16 w + 4 (l / 16) + i.
template <int DT>
using Part = Eight<DT>[4];

// Codes of 4 rows of column e.
template <int DT, int TYPE, bool ANY>
__device__ __forceinline__ uint32_t col_codes(const Eight<DT> (&v)[4], int e, int s) {
    if constexpr (DT == ZS_BF16) {
        const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
        return four_codes<TYPE, ANY>(__builtin_amdgcn_perm(v[1].w[e / 2], v[0].w[e / 2], sel),
                                     __builtin_amdgcn_perm(v[3].w[e / 2], v[2].w[e / 2], sel), s);
    } else {
        return four_codes<TYPE, ANY>(v[0].f[e], v[1].f[e], v[2].f[e], v[3].f[e], s);
    }
}

template <int DT, int BR, int TYPE, bool ANY>
__device__ __forceinline__ void put_rows(const F8Quant& q, const Part<DT>& x, const int (&s)[4],
                                         int64_t row0, int64_t tc, int cg) {
    const int64_t blocks = f8_ceil(q.cols, kT);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row0 + i;
        const u32x2 w = eight_codes<DT, TYPE, ANY>(x[i], s[i]);
        if (r >= q.rows) continue;
        *global<g_u32x2a>(q.out.codes + r * q.out.ld + tc * kT + 8 * cg) = w;
        if (BR == 1 && cg < 4) put_scale(q.out, r, tc, blocks, cg, s[i]);
    }
}
template <int DT, int TYPE, bool ANY>
__device__ __forceinline__ void stage_cols(const Part<DT>& x, const int (&s)[8], int wave, int cg,
                                           int rq, Shared& sh) {
    // word (column, 4 rows): the 16-byte pieces of a column's 128 are permuted by its number
    // over 8, so that the 16 columns that a wavefront writes at once fall on other banks
#pragma unroll
    for (int e = 0; e < 8; ++e)
        sh.codes[(8 * cg + e) * 32 + 4 * (wave ^ (cg & 7)) + rq] =
            col_codes<DT, TYPE, ANY>(x, e, s[e]);
}

// One tile. BR = 1: a block for each row (column, transposed) of the tile, BR = 128: one.
// Special blocks are rare: a wavefront without one converts by the instruction alone.
template <int DT, int BR, class Src>
__device__ __forceinline__ void quant_tile(const F8Quant& q, const Src& src, int64_t tr,
                                           int64_t tc, Shared& sh) {
    const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
    const int cg = lane & 15, rq = lane >> 4;
    const int64_t r0 = tr * kT, row0 = r0 + 16 * wave + 4 * rq, c = tc * kT + 8 * cg;
    const int live = q.cols - c >= 8 ? 8 : (q.cols > c ? int(q.cols - c) : 0);
    Part<DT> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (row0 + i < q.rows && live > 0) x[i] = src.template get<DT>(row0 + i, c, live);
        else x[i] = Eight<DT>{};
    }
    uint32_t whole = 0;
    if constexpr (BR == 128) {
#pragma unroll
        for (int i = 0; i < 4; ++i) whole = max_u(whole, top_bits<DT>(x[i]));
        whole = col_max(row_max(whole));
        if (lane == 0) sh.whole[wave] = whole;
        __syncthreads();
        whole = max_of(sh.whole, 1);
    }
    if (q.out.codes != nullptr) {
        const int type = q.out.type;
        int s[4];
        bool special = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = BR == 128 ? whole : row_max(top_bits<DT>(x[i]));
            s[i] = scale_of(u, type);
            special |= is_special(u, s[i]);
        }
        if (__any(special)) {
            if (type == ZS_E4M3) put_rows<DT, BR, ZS_E4M3, true>(q, x, s, row0, tc, cg);
            else put_rows<DT, BR, ZS_E5M2, true>(q, x, s, row0, tc, cg);
        } else {
            if (type == ZS_E4M3) put_rows<DT, BR, ZS_E4M3, false>(q, x, s, row0, tc, cg);
            else put_rows<DT, BR, ZS_E5M2, false>(q, x, s, row0, tc, cg);
        }
        if (BR == 128 && threadIdx.x < 4)
            put_scale(q.out, tr, tc, f8_ceil(q.cols, kT), int(threadIdx.x), scale_of(whole, type));
    }
    if (q.out_t.codes == nullptr) return;
    const int type = q.out_t.type;
    const int64_t blocks_r = f8_ceil(q.rows, kT);
    int s[8];
    bool special = false;
    if constexpr (BR == 1) {
        // a column's largest magnitude: of the lane's 4 rows, the wavefront's 16, all 128
        if constexpr (DT == ZS_BF16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u16x2 u = mags(x[0].w[k]);
#pragma unroll
                for (int i = 1; i < 4; ++i)
                    u = __builtin_elementwise_max(u, mags(x[i].w[k]));
                const uint32_t two = col_max_pair(__builtin_bit_cast(uint32_t, u));
                if (rq == 0) {
                    sh.top[wave][8 * cg + 2 * k] = two << 16;
                    sh.top[wave][8 * cg + 2 * k + 1] = two & 0xffff0000u;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t u = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    u = max_u(u, __float_as_uint(x[i].f[e]) & 0x7fffffffu);
                u = col_max(u);
                if (rq == 0) sh.top[wave][8 * cg + e] = u;
            }
        }
        __syncthreads();
        // one thread a column joins the wavefronts' maxima; bit 8 of its word: a special block
        if (threadIdx.x < kT) {
            const uint32_t u = max_of(&sh.top[0][threadIdx.x], kT);
            const int mine = scale_of(u, type);
            sh.scale[threadIdx.x] = mine | (is_special(u, mine) ? 256 : 0);
            const int64_t col = tc * kT + int(threadIdx.x);
            if (col < q.cols) {
#pragma unroll
                for (int k = 0; k < 4; ++k) put_scale(q.out_t, col, tr, blocks_r, k, mine);
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int w = sh.scale[8 * cg + e];
            s[e] = w & 255;
            special |= w > 255;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = scale_of(whole, type);
        special = is_special(whole, s[0]);
        if (threadIdx.x < 4)
            put_scale(q.out_t, tc, tr, blocks_r, int(threadIdx.x), scale_of(whole, type));
    }
    if (__any(special)) {
        if (type == ZS_E4M3) stage_cols<DT, ZS_E4M3, true>(x, s, wave, cg, rq, sh);
        else stage_cols<DT, ZS_E5M2, true>(x, s, wave, cg, rq, sh);
    } else {
        if (type == ZS_E4M3) stage_cols<DT, ZS_E4M3, false>(x, s, wave, cg, rq, sh);
        else stage_cols<DT, ZS_E5M2, false>(x, s, wave, cg, rq, sh);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16 / kWaves; ++k) {
        const int col = 8 * kWaves * k + int(threadIdx.x) / 8, piece = int(threadIdx.x) % 8;
        if (tc * kT + col < q.cols) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(
                &sh.codes[col * 32 + 4 * (piece ^ ((col >> 3) & 7))]);
            *global<g_u32x4a>(q.out_t.codes + (tc * kT + col) * q.out_t.ld + r0 + 16 * piece) = w;
        }
    }
}

// One matrix, or (tiles2 > 0) two in one launch.
template <int DT, int BR>
__global__ __launch_bounds__(kTileThreads, 4) void quantize_kernel(
    F8Quant one, F8Quant two, uint32_t tiles1, uint32_t tiles2) {
    __shared__ Shared sh;
    for (uint32_t t = blockIdx.x; t < tiles1 + tiles2; t += gridDim.x) {
        const F8Quant& q = t < tiles1 ? one : two;
        const uint32_t in = t < tiles1 ? t : t - tiles1;
        const uint32_t tiles_c = uint32_t(f8_ceil(q.cols, kT));
        const Strided src{q.x, q.ldx};
        quant_tile<DT, BR>(q, src, in / tiles_c, in % tiles_c, sh);
        __syncthreads();
    }
}

template <int DT, int BR>
__global__ __launch_bounds__(kTileThreads, 4) void gather_kernel(F8Quant q, F8Shards s) {
    __shared__ Shared sh;
    const uint32_t tiles_c = uint32_t(f8_ceil(q.cols, kT));
    const uint32_t tiles = tiles_c * uint32_t(f8_ceil(q.rows, kT));  // checked: below 2^31
    const Sharded src{&s, q.cols};
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        quant_tile<DT, BR>(q, src, t / tiles_c, t % tiles_c, sh);
        __syncthreads();
    }
}

// Value of a code under scale byte s, as fp32.
template <int TYPE>
__device__ __forceinline__ f32x2 two_values(uint32_t w, bool hi) {
    if constexpr (TYPE == ZS_E4M3)
        return hi ? __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true)
                  : __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
    else
        return hi ? __builtin_amdgcn_cvt_pk_f32_bf8(int(w), true)
                  : __builtin_amdgcn_cvt_pk_f32_bf8(int(w), false);
}

// Tiles of 64 x 128; a lane takes the codes of 16 bytes of values (8 bf16 or 4 fp32), so
// that a wavefront's store covers whole runs of its rows.
template <int TYPE, int DT>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int shift,
    int64_t rows, int64_t cols, int64_t ld, int64_t lds, void* __restrict__ out, int64_t ldo) {
    constexpr int E = DT == ZS_BF16 ? 8 : 4, kLanes = kT / E, kRows = kThreads / kLanes;
    constexpr int kTileRows = 64;
    const uint32_t tiles_c = uint32_t(f8_ceil(cols, kT));
    const uint32_t tiles = tiles_c * uint32_t(f8_ceil(rows, kTileRows));
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t tr = t / tiles_c, tc = t % tiles_c;
        const int64_t c = tc * kT + E * (int(threadIdx.x) % kLanes);
        uint32_t w[kTileRows / kRows][E / 4];
        int s[kTileRows / kRows];
#pragma unroll
        for (int k = 0; k < kTileRows / kRows; ++k) {
            const int64_t r = tr * kTileRows + k * kRows + int(threadIdx.x) / kLanes;
            if (r >= rows) continue;
            const g_u32a* p = global<const g_u32a>(codes + r * ld + c);
#pragma unroll
            for (int j = 0; j < E / 4; ++j) w[k][j] = p[j];
            s[k] = global<const g_u8>(scales)[(r >> shift) * lds + tc];
        }
#pragma unroll
        for (int k = 0; k < kTileRows / kRows; ++k) {
            const int64_t r = tr * kTileRows + k * kRows + int(threadIdx.x) / kLanes;
            if (r >= rows || c >= cols) continue;
            float y[E];
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const f32x2 v = two_values<TYPE>(w[k][j / 2], j & 1);
                y[2 * j] = v[0], y[2 * j + 1] = v[1];
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
                y[j] = __builtin_ldexpf(y[j], s[k] - 127);
                if (s[k] == 255) y[j] = __uint_as_float(0x7fc00000u);
            }
            const int64_t at = r * ldo + c;
            if (c + E <= cols) {
                if constexpr (DT == ZS_BF16)
                    __builtin_nontemporal_store(
                        u32x4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                              pack_bf16(y[6], y[7])},
                        reinterpret_cast<g_u32x4*>(global<g_u16>(out) + at));
                else
                    __builtin_nontemporal_store(
                        f32x4{y[0], y[1], y[2], y[3]},
                        reinterpret_cast<g_f32x4*>(global<g_f32>(out) + at));
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if (c + j >= cols) continue;
                    if constexpr (DT == ZS_BF16)
                        global<g_u16>(out)[at + j] = uint16_t(pack_bf16(y[j], 0.0f));
                    else
                        global<g_f32>(out)[at + j] = y[j];
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_quantize_f8(const F8Quant& q, int block_rows, hipStream_t stream) {
    const uint32_t tiles = uint32_t(f8_tiles(q.rows, q.cols));  // checked: below 2^31
    const dim3 grid(unsigned(f8_quant_grid(tiles)));
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kTileThreads), 0, stream, q, q, tiles, 0u);
    };
    if (q.dtype == ZS_BF16) {
        if (block_rows == 1) go(quantize_kernel<ZS_BF16, 1>);
        else go(quantize_kernel<ZS_BF16, 128>);
    } else {
        if (block_rows == 1) go(quantize_kernel<ZS_F32, 1>);
        else go(quantize_kernel<ZS_F32, 128>);
    }
    return hipGetLastError();
}

hipError_t launch_quantize2_f8(const F8Quant& one, const F8Quant& two, hipStream_t stream) {
    const uint32_t a = uint32_t(f8_tiles(one.rows, one.cols)),
                   b = uint32_t(f8_tiles(two.rows, two.cols));  // checked: each below 2^30
    const dim3 grid(unsigned(f8_quant_grid(int64_t(a) + b)));
    if (one.dtype == ZS_BF16)
        hipLaunchKernelGGL((quantize_kernel<ZS_BF16, 1>), grid, dim3(kTileThreads), 0, stream, one, two,
                           a, b);
    else
        hipLaunchKernelGGL((quantize_kernel<ZS_F32, 1>), grid, dim3(kTileThreads), 0, stream, one, two,
                           a, b);
    return hipGetLastError();
}

hipError_t launch_gather_f8(const F8Quant& q, const F8Shards& src, int block_rows,
                            hipStream_t stream) {
    const dim3 grid(unsigned(f8_quant_grid(f8_tiles(q.rows, q.cols))));
    if (q.dtype == ZS_BF16) {
        if (block_rows == 1)
            hipLaunchKernelGGL((gather_kernel<ZS_BF16, 1>), grid, dim3(kTileThreads), 0, stream, q, src);
        else
            hipLaunchKernelGGL((gather_kernel<ZS_BF16, 128>), grid, dim3(kTileThreads), 0, stream, q,
                               src);
    } else {
        if (block_rows == 1)
            hipLaunchKernelGGL((gather_kernel<ZS_F32, 1>), grid, dim3(kTileThreads), 0, stream, q, src);
        else
            hipLaunchKernelGGL((gather_kernel<ZS_F32, 128>), grid, dim3(kTileThreads), 0, stream, q,
                               src);
    }
    return hipGetLastError();
}

hipError_t launch_dequantize_f8(const uint8_t* codes, const uint8_t* scales, int block_rows,
                                int64_t rows, int64_t cols, int type, int dtype, void* out,
                                int64_t ldo, hipStream_t stream) {
    const int64_t ld = f8_ld(cols), lds = f8_lds(cols);
    const int shift = block_rows == 1 ? 0 : 7;
    const dim3 grid(unsigned(f8_values_grid(rows, cols)));
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, codes, scales, shift, rows,
                           cols, ld, lds, out, ldo);
    };
    if (type == ZS_E4M3) {
        if (dtype == ZS_BF16) go(dequantize_kernel<ZS_E4M3, ZS_BF16>);
        else go(dequantize_kernel<ZS_E4M3, ZS_F32>);
    } else {
        if (dtype == ZS_BF16) go(dequantize_kernel<ZS_E5M2, ZS_BF16>);
        else go(dequantize_kernel<ZS_E5M2, ZS_F32>);
    }
    return hipGetLastError();
}

}  // namespace zs

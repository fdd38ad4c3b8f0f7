// Products of block-scaled 8-bit matrices, C[m, n] = sum_k a[m, k] b[n, k], for gfx950.
//
// A workgroup sums a TM x TN tile of C over its part of K in steps of 128, one block of
// both operands: their codes go from memory straight to LDS (16 bytes a lane, two buffers,
// the next step's under way while this one is multiplied), and every wavefront multiplies
// its PM x PN part from there. Both operands lie along K, so that all accesses are 16-byte
// pieces of 128-byte rows; piece j of row r stands at j ^ (r mod 8) of its row in LDS, so
// that the 16 rows that a wavefront reads at once fall on all banks.
//
// C in bf16: v_mfma_scale_f32_16x16x128_f8f6f4 multiplies a whole block with both scale
// bytes. Of 8 neighbouring products it drops what is below 2^-13 of the largest one's power
// of two (measured; the sums of the eights are added in fp32): on normal data 2^-16 of the
// result, 2^7 below the rounding to bf16. C in fp32 (EXACT): the codes, times their scales, become bf16
// exactly and v_mfma_f32_16x16x32_bf16 sums them in fp32, at a quarter of the rate.
//
// The matrix instruction's first operand is b and its second a: a lane then holds 4
// neighbouring columns n of C.

#include "zs_f8.h"
#include "zs_math.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = kBlockThreads;
constexpr int kB = kF8Block;

#define ZS_GLOBAL __attribute__((address_space(1)))
#define ZS_LDS __attribute__((address_space(3)))
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef ZS_GLOBAL f32x4_u g_f32x4;
typedef ZS_GLOBAL u32x2_u g_u32x2;
typedef ZS_GLOBAL uint8_t g_u8;
typedef ZS_GLOBAL uint16_t g_u16;
typedef ZS_GLOBAL uint32_t g_u32;
typedef ZS_GLOBAL uint64_t g_u64;
typedef ZS_GLOBAL float g_f32;

template <typename G, typename P>
__device__ __forceinline__ G* global(P* p) {
    return reinterpret_cast<G*>(reinterpret_cast<uintptr_t>(p));
}

// Codes of one step of ROWS rows from row `first` on, to LDS. Rows past the operand's last
// are its last again: what they give is not stored.
template <int ROWS>
__device__ __forceinline__ void stage(const F8Operand& x, int64_t first, int block, uint8_t* lds) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int piece = (lane & 7) ^ (lane >> 3);
#pragma unroll
    for (int k = 0; k < ROWS / 32; ++k) {
        const int part = k * 4 + wave;  // of 8 rows
        int64_t r = first + part * 8 + (lane >> 3);
        r = r < x.rows ? r : x.rows - 1;
        const uint8_t* p = x.codes + r * x.ld + int64_t(block) * kB + piece * 16;
        __builtin_amdgcn_global_load_lds(global<ZS_GLOBAL void>(const_cast<uint8_t*>(p)),
                                         (ZS_LDS void*)(lds + part * 1024), 16, 0, 0);
    }
}

// A lane's 32 codes of one row of a step.
__device__ __forceinline__ i32x8 fragment(const uint8_t* lds, int row0) {
    const int lane = int(threadIdx.x) & 63;
    const int row = row0 + (lane & 15), g = lane >> 4;
    const i32x4 a = *reinterpret_cast<const i32x4*>(lds + row * kB + (((2 * g) ^ (row & 7)) * 16));
    const i32x4 b = *reinterpret_cast<const i32x4*>(lds + row * kB + (((2 * g + 1) ^ (row & 7)) * 16));
    return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The word with a lane's row's scale bytes of 4 steps.
__device__ __forceinline__ uint32_t scale_word(const F8Operand& x, int64_t row, int block) {
    row = row < x.rows ? row : x.rows - 1;
    return *global<const g_u32>(x.scales + (row >> x.shift) * x.lds + (block & ~3));
}

__device__ __forceinline__ float scale_value(uint32_t s) {
    s &= 255u;
    return s == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(s == 0 ? 0x400000u : s << 23);
}

// 8 codes, words w0 and w1, as bf16 times the scale.
template <int TYPE>
__device__ __forceinline__ bf16x8 widen(int w0, int w1, float two) {
    bf16x2 h[4];
    if constexpr (TYPE == ZS_E4M3) {
        h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(uint32_t(w0), two, false);
        h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(uint32_t(w0), two, true);
        h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(uint32_t(w1), two, false);
        h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(uint32_t(w1), two, true);
    } else {
        h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(uint32_t(w0), two, false);
        h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(uint32_t(w0), two, true);
        h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(uint32_t(w1), two, false);
        h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(uint32_t(w1), two, true);
    }
    return bf16x8{h[0][0], h[0][1], h[1][0], h[1][1], h[2][0], h[2][1], h[3][0], h[3][1]};
}

template <int TYPE>
constexpr int kFormat = TYPE == ZS_E4M3 ? 0 : 1;

// 4 neighbouring elements of a row of C.
template <int DT>
__device__ __forceinline__ void put4(const F8Product& p, int64_t m, int64_t n, int64_t N, f32x4 v) {
    const int64_t at = m * p.ldc + n;
    const int live = N - n >= 4 ? 4 : int(N - n);
    if constexpr (DT == ZS_BF16) {
        g_u16* c = global<g_u16>(p.c) + at;
        if (p.accumulate) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) v[e] += __uint_as_float(uint32_t(c[e]) << 16);
        }
        const u32x2 w{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        if (live == 4) {
            *reinterpret_cast<g_u32x2*>(c) = w;
            return;
        }
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < live) c[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
    } else {
        g_f32* c = global<g_f32>(p.c) + at;
        if (p.accumulate) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < live) v[e] += c[e];
        }
        if (live == 4) {
            *reinterpret_cast<g_f32x4*>(c) = v;
            return;
        }
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < live) c[e] = v[e];
    }
}

// TM x TN of C by 4 wavefronts, 2 x 2.
template <int TM, int TN, int TA, int TB, int DT>
__global__ __launch_bounds__(kThreads) void matmul_kernel(F8Product p) {
    constexpr bool EXACT = DT == ZS_F32;
    constexpr int PM = TM / 2, PN = TN / 2, MI = PM / 16, NI = PN / 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][(TM + TN) * kB];
    __shared__ bool last;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int split = int(blockIdx.x % unsigned(p.splits));
    const int tile = int(blockIdx.x / unsigned(p.splits));
    const int64_t m0 = int64_t(tile / p.tiles_n) * TM, n0 = int64_t(tile % p.tiles_n) * TN;
    const int wm = (wave & 1) * PM, wn = (wave >> 1) * PN;
    const int k0 = int(int64_t(p.blocks) * split / p.splits);
    const int k1 = int(int64_t(p.blocks) * (split + 1) / p.splits);

    f32x4 acc[NI][MI] = {};
    uint32_t sa[MI], sb[NI];
    if (k0 < k1) {
        stage<TM>(p.a, m0, k0, lds[0]);
        stage<TN>(p.b, n0, k0, lds[0] + TM * kB);
    }
    for (int k = k0; k < k1; ++k) {
        uint8_t* const now = lds[(k - k0) & 1];
        uint8_t* const next = lds[(k - k0 + 1) & 1];
        if (k == k0 || (k & 3) == 0) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
                sa[i] = scale_word(p.a, m0 + wm + 16 * i + (lane & 15), k) >> (8 * (k & 3));
#pragma unroll
            for (int i = 0; i < NI; ++i)
                sb[i] = scale_word(p.b, n0 + wn + 16 * i + (lane & 15), k) >> (8 * (k & 3));
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();  // this step's codes are there, and the other buffer is read out
        if (k + 1 < k1) {
            stage<TM>(p.a, m0, k + 1, next);
            stage<TN>(p.b, n0, k + 1, next + TM * kB);
        }
        i32x8 a[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) a[i] = fragment(now, wm + 16 * i);
        if constexpr (!EXACT) {
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const i32x8 b = fragment(now + TM * kB, wn + 16 * j);
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        b, a[i], acc[j][i], kFormat<TB>, kFormat<TA>, 0, int(sb[j]), 0, int(sa[i]));
            }
        } else {
            i32x8 b[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j) b[j] = fragment(now + TM * kB, wn + 16 * j);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 h[MI];
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    h[i] = widen<TA>(a[i][2 * q], a[i][2 * q + 1], scale_value(sa[i]));
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const bf16x8 g = widen<TB>(b[j][2 * q], b[j][2 * q + 1], scale_value(sb[j]));
#pragma unroll
                    for (int i = 0; i < MI; ++i)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(g, h[i], acc[j][i], 0, 0, 0);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] >>= 8;
#pragma unroll
        for (int i = 0; i < NI; ++i) sb[i] >>= 8;
    }

    if (p.splits > 1) {
        // partial sums as the lanes hold them, written through to memory that all XCDs share;
        // the workgroup that counts in last adds them in their order
        typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
        uint64_t* const mine = reinterpret_cast<uint64_t*>(p.partial) +
                               (int64_t(tile) * p.splits + split) * (TM * TN / 2) +
                               (wave * NI * MI * 64 + lane) * 2;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const u64x2 v = __builtin_bit_cast(u64x2, acc[j][i]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    __hip_atomic_store(&mine[(j * MI + i) * 128 + e], v[e], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t* const n = p.counts + tile;
            last = __hip_atomic_fetch_add(n, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 ==
                   uint32_t(p.splits);
            if (last) __hip_atomic_store(n, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!last) return;
        const uint64_t* from = reinterpret_cast<const uint64_t*>(p.partial) +
                               int64_t(tile) * p.splits * (TM * TN / 2) +
                               (wave * NI * MI * 64 + lane) * 2;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i) acc[j][i] = f32x4{0, 0, 0, 0};
        for (int s = 0; s < p.splits; ++s, from += TM * TN / 2) {
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    u64x2 v;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        v[e] = __hip_atomic_load(&from[(j * MI + i) * 128 + e], __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT);
                    acc[j][i] += __builtin_bit_cast(f32x4, v);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + wm + 16 * i + (lane & 15);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t n = n0 + wn + 16 * j + 4 * (lane >> 4);
            if (m < p.a.rows && n < p.b.rows) put4<DT>(p, m, n, p.b.rows, acc[j][i]);
        }
    }
}

template <int TM, int TN, int TA, int TB>
void launch_tile(const F8Product& p, int dtype, hipStream_t stream) {
    const dim3 grid(unsigned(int64_t(p.tiles_m) * p.tiles_n * p.splits));
    if (dtype == ZS_BF16)
        hipLaunchKernelGGL((matmul_kernel<TM, TN, TA, TB, ZS_BF16>), grid, dim3(kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((matmul_kernel<TM, TN, TA, TB, ZS_F32>), grid, dim3(kThreads), 0, stream, p);
}

template <int TA, int TB>
void launch_types(const F8Product& p, const F8Plan& plan, int dtype, hipStream_t stream) {
    if (plan.tm == 128) launch_tile<128, 128, TA, TB>(p, dtype, stream);
    else launch_tile<64, 64, TA, TB>(p, dtype, stream);
}

}  // namespace

hipError_t launch_matmul_f8(const F8Product& p, const F8Plan& plan, int type_a, int type_b,
                            int dtype, hipStream_t stream) {
    if (type_a == ZS_E4M3) {
        if (type_b == ZS_E4M3) launch_types<ZS_E4M3, ZS_E4M3>(p, plan, dtype, stream);
        else launch_types<ZS_E4M3, ZS_E5M2>(p, plan, dtype, stream);
    } else {
        if (type_b == ZS_E4M3) launch_types<ZS_E5M2, ZS_E4M3>(p, plan, dtype, stream);
        else launch_types<ZS_E5M2, ZS_E5M2>(p, plan, dtype, stream);
    }
    return hipGetLastError();
}

}  // namespace zs

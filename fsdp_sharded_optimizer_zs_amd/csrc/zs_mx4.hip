// Microscaled 4-bit shards for gfx950: quantisation of a bf16 or fp32 shard, and the
// gather that rebuilds a unit from such shards.
//
// Both stream once over their data and are bound by HBM: the quantiser reads 2 or 4
// bytes an element and writes 0.53, the gather reads 0.53 and writes 2 or 4. A lane
// takes 8 consecutive elements, one 32-bit word of codes; 4 lanes share a block of
// 32 and its scale byte.
//
// An element's 3 magnitude bits (2 of exponent, 1 of mantissa) are the top of an fp32
// pattern: the value 2^(s-127) * e2m1 is float_of_bits(c << 22) * 2^(s - 1), whose
// subnormal 0.5 is fp32's own subnormal, so decoding is a shift and an exponent
// adjustment and encoding rounds the pattern at bit 22.

#include "zs_multi.h"
#include "zs_math.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = kBlockThreads;
constexpr int kVec = 8;  // elements per lane

#define ZS_GLOBAL __attribute__((address_space(1)))
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// vectors at element alignment: a shard, or its slot of the unit, may start at any
// element, and gfx950 accesses it with the same one wide instruction
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_u __attribute__((aligned(1)));
typedef ZS_GLOBAL f32x4_u g_f32x4;
typedef ZS_GLOBAL u32x4_u g_u32x4;
typedef ZS_GLOBAL u32_u g_u32;
typedef ZS_GLOBAL uint8_t g_u8;
typedef ZS_GLOBAL uint16_t g_u16;
typedef ZS_GLOBAL float g_f32;

template <typename G, typename P>
__device__ __forceinline__ G* global(P* p) {
    return reinterpret_cast<G*>(reinterpret_cast<uintptr_t>(p));
}

template <int DT>
__device__ __forceinline__ void load8(const void* src, int64_t i, int live, float (&x)[kVec]) {
    if constexpr (DT == ZS_BF16) {
        const g_u16* s = global<const g_u16>(src) + i;
        if (live == kVec) {
            const u32x4 h = __builtin_nontemporal_load(reinterpret_cast<const g_u32x4*>(s));
#pragma unroll
            for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(h[k]), x[2 * k + 1] = bf16_hi(h[k]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                x[e] = e < live ? __uint_as_float(uint32_t(s[e]) << 16) : 0.0f;
        }
    } else {
        const g_f32* s = global<const g_f32>(src) + i;
        if (live == kVec) {
            const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(s));
            const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(s + 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = a[k], x[4 + k] = b[k];
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] = e < live ? s[e] : 0.0f;
        }
    }
}

// Largest u of the 4 lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t u) {
    uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0xb1, 0xf, 0xf, true));  // 1,0,3,2
    u = u > o ? u : o;
    o = uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x4e, 0xf, 0xf, true));           // 2,3,0,1
    return u > o ? u : o;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ src, int64_t S,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    const int64_t nv = (S + kVec - 1) / kVec;
    const int lane = int(threadIdx.x) & 63;
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    // every lane of a wavefront makes the same trips: quads exchange across lanes
    for (int64_t v0 = int64_t(blockIdx.x) * kThreads + (threadIdx.x - lane); v0 < nv; v0 += stride) {
        const int64_t v = v0 + lane;
        const int64_t i = v * kVec;
        const int live = i >= S ? 0 : (S - i >= kVec ? kVec : int(S - i));
        float x[kVec];
        load8<DT>(src, i, live, x);
        uint32_t u = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
            u = u > b ? u : b;
        }
        u = quad_max(u);
        int s = int(u >> 23) - 2;
        s = s > 0 ? s : 0;
        uint32_t w = 0;
        if (u >= 0x7f800000u) {
            s = 255;
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const uint32_t b =
                    __float_as_uint(__builtin_ldexpf(__builtin_fabsf(x[e]), 1 - s));
                uint32_t c = (b + 0x1fffffu + ((b >> 22) & 1u)) >> 22;
                c = c < 7u ? c : 7u;
                w |= (c | ((__float_as_uint(x[e]) >> 31) << 3)) << (4 * e);
            }
        }
        if (live == kVec) {
            __builtin_nontemporal_store(w, reinterpret_cast<g_u32*>(global<g_u8>(codes) + i / 2));
        } else {
            // x is +0 past the end, so the last half byte of an odd shard is 0
#pragma unroll
            for (int k = 0; k < kVec / 2; ++k)
                if (2 * k < live) global<g_u8>(codes)[i / 2 + k] = uint8_t(w >> (8 * k));
        }
        if ((lane & 3) == 0 && live > 0) global<g_u8>(scales)[v >> 2] = uint8_t(s);
    }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void gather_mx4_kernel(PtrPack codes, PtrPack scales,
                                                              int64_t S, void* __restrict__ flat) {
    const int r = int(blockIdx.y);
    const g_u8* cs = global<const g_u8>(static_cast<const uint8_t*>(codes.p[r]));
    const g_u8* ss = global<const g_u8>(static_cast<const uint8_t*>(scales.p[r]));
    const int64_t nv = (S + kVec - 1) / kVec;
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t v = int64_t(blockIdx.x) * kThreads + threadIdx.x; v < nv; v += stride) {
        const int64_t i = v * kVec;
        const int live = S - i >= kVec ? kVec : int(S - i);
        uint32_t w = 0;
        if (live == kVec) {
            w = __builtin_nontemporal_load(reinterpret_cast<const g_u32*>(cs + i / 2));
        } else {
#pragma unroll
            for (int k = 0; k < kVec / 2; ++k)
                if (2 * k < live) w |= uint32_t(cs[i / 2 + k]) << (8 * k);
        }
        const int s = ss[v >> 2];
        float x[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint32_t c = w >> (4 * e);
            x[e] = __builtin_ldexpf(__uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)), s - 1);
            if (s == 255) x[e] = __uint_as_float(0x7fc00000u);
        }
        const int64_t o = int64_t(r) * S + i;
        if constexpr (DT == ZS_BF16) {
            g_u16* d = global<g_u16>(static_cast<uint16_t*>(flat)) + o;
            if (live == kVec) {
                u32x4 h;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[k] = f32_to_bf16(x[2 * k]) | (f32_to_bf16(x[2 * k + 1]) << 16);
                __builtin_nontemporal_store(h, reinterpret_cast<g_u32x4*>(d));
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e < live) d[e] = uint16_t(f32_to_bf16(x[e]));
            }
        } else {
            g_f32* d = global<g_f32>(static_cast<float*>(flat)) + o;
            if (live == kVec) {
                __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]},
                                            reinterpret_cast<g_f32x4*>(d));
                __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]},
                                            reinterpret_cast<g_f32x4*>(d + 4));
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e < live) d[e] = x[e];
            }
        }
    }
}

}  // namespace

hipError_t launch_quantize_mx4(const void* src, int dtype, int64_t S, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream) {
    const dim3 grid(unsigned(quantize_mx4_grid(S)));
    if (dtype == ZS_BF16)
        hipLaunchKernelGGL((quantize_kernel<ZS_BF16>), grid, dim3(kThreads), 0, stream, src, S,
                           codes, scales);
    else
        hipLaunchKernelGGL((quantize_kernel<ZS_F32>), grid, dim3(kThreads), 0, stream, src, S,
                           codes, scales);
    return hipGetLastError();
}

hipError_t launch_gather_mx4(const PtrPack& codes, const PtrPack& scales, int D, int64_t S,
                             int dtype, void* flat, hipStream_t stream) {
    const dim3 grid(unsigned(gather_mx4_grid(S, D)), unsigned(D));
    if (dtype == ZS_BF16)
        hipLaunchKernelGGL((gather_mx4_kernel<ZS_BF16>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, flat);
    else
        hipLaunchKernelGGL((gather_mx4_kernel<ZS_F32>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, flat);
    return hipGetLastError();
}

}  // namespace zs

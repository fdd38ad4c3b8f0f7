// Microscaled 4-bit shards for gfx950: quantisation of a bf16 or fp32 shard, and the
// gather that rebuilds a unit from such shards.
//
// Both stream once over their data and are bound by HBM: the quantiser reads 2 or 4
// bytes an element and writes 0.53, the gather reads 0.53 and writes 2 or 4. A lane
// takes 8 consecutive elements at a time, one 32-bit word of codes, and kMx4Unroll such
// groups, a workgroup apart, whose loads are all ahead of their use; 4 lanes share a
// block of 32 and its scale byte.
//
// Two elements are converted by one instruction of gfx950 (v_cvt_scalef32_pk_*_fp4),
// which takes 2^(s-127) as a float. For s = 0 that float would be subnormal, and s = 255
// is NaN: those blocks (largest magnitude below 2^-124, or not finite) are converted
// with integer operations instead. There an element's 3 magnitude bits (2 of exponent, 1
// of mantissa) are the top of an fp32 pattern: 2^(s-127) * e2m1 is float_of_bits(c << 22)
// * 2^(s - 1), whose subnormal 0.5 is fp32's own subnormal, so decoding is a shift and an
// exponent adjustment and encoding rounds the pattern at bit 22.

#include "zs_multi.h"
#include "zs_math.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = kBlockThreads;
constexpr int kVec = 8;  // elements of a lane's group

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

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// A lane's 8 elements: bf16 as 4 words of pairs, fp32 as 8 words.
template <int DT>
struct Group {
    static constexpr int words = DT == ZS_BF16 ? 4 : 8;
    uint32_t w[words];
};

template <int DT>
__device__ __forceinline__ void load_group(const void* src, int64_t i, Group<DT>& x) {
    if constexpr (DT == ZS_BF16) {
        const u32x4 h = __builtin_nontemporal_load(
            reinterpret_cast<const g_u32x4*>(global<const g_u16>(src) + i));
#pragma unroll
        for (int k = 0; k < 4; ++k) x.w[k] = h[k];
    } else {
        const g_f32* s = global<const g_f32>(src) + i;
        const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(s));
        const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(s + 4));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x.w[k] = __float_as_uint(a[k]), x.w[4 + k] = __float_as_uint(b[k]);
    }
}
// The first `live` of them, the others +0.
template <int DT>
__device__ __forceinline__ void load_group_part(const void* src, int64_t i, int live,
                                                Group<DT>& x) {
#pragma unroll
    for (int k = 0; k < Group<DT>::words; ++k) x.w[k] = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        if (e >= live) continue;
        if constexpr (DT == ZS_BF16)
            x.w[e / 2] |= uint32_t(global<const g_u16>(src)[i + e]) << (16 * (e & 1));
        else
            x.w[e] = __float_as_uint(global<const g_f32>(src)[i + e]);
    }
}
template <int DT>
__device__ __forceinline__ float value_of(const Group<DT>& x, int e) {
    if constexpr (DT == ZS_BF16) return e & 1 ? bf16_hi(x.w[e / 2]) : bf16_lo(x.w[e / 2]);
    else return __uint_as_float(x.w[e]);
}

// The fp32 bits of the largest magnitude of a lane's 8 elements (as unsigned numbers:
// infinity and NaN above every number).
template <int DT>
__device__ __forceinline__ uint32_t top_bits(const Group<DT>& x) {
    if constexpr (DT == ZS_BF16) {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 u{0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            u = __builtin_elementwise_max(u, __builtin_bit_cast(u16x2, x.w[k] & 0x7fff7fffu));
        return uint32_t(u[0] > u[1] ? u[0] : u[1]) << 16;
    } else {
        uint32_t u = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = x.w[k] & 0x7fffffffu;
            u = u > b ? u : b;
        }
        return u;
    }
}

// Largest u of the 4 lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t u) {
    uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0xb1, 0xf, 0xf, true));  // 1,0,3,2
    u = u > o ? u : o;
    o = uint32_t(__builtin_amdgcn_mov_dpp(int(u), 0x4e, 0xf, 0xf, true));           // 2,3,0,1
    return u > o ? u : o;
}

// Scale byte and word of codes of a lane's group. Every lane of the quad calls it.
template <int DT>
__device__ __forceinline__ uint32_t encode(const Group<DT>& x, int* scale) {
    const uint32_t u = quad_max(top_bits<DT>(x));
    int s = int(u >> 23) - 2;
    s = u >= 0x7f800000u ? 255 : (s > 0 ? s : 0);
    *scale = s;
    uint32_t w = 0;
    if (s != 0 && s != 255) {
        const float two = __uint_as_float(uint32_t(s) << 23);
        if constexpr (DT == ZS_BF16) {
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
                w, __builtin_bit_cast(bf16x2, x.w[0]), two, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
                w, __builtin_bit_cast(bf16x2, x.w[1]), two, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
                w, __builtin_bit_cast(bf16x2, x.w[2]), two, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(
                w, __builtin_bit_cast(bf16x2, x.w[3]), two, 3);
        } else {
            const auto f = [&](int k) { return __uint_as_float(x.w[k]); };
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(0), f(1), two, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(2), f(3), two, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(4), f(5), two, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(6), f(7), two, 3);
        }
    } else if (s == 0) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const float y = value_of<DT>(x, e);
            const uint32_t b = __float_as_uint(__builtin_ldexpf(__builtin_fabsf(y), 1 - s));
            uint32_t c = (b + 0x1fffffu + ((b >> 22) & 1u)) >> 22;
            c = c < 7u ? c : 7u;
            w |= (c | ((__float_as_uint(y) >> 31) << 3)) << (4 * e);
        }
    }
    return w;
}

// A bf16 shard of 25.3M elements: 12.4 us, 5.2 TB/s with the launch's start and end (one
// group a lane and integer conversions: about 18).
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ src, int64_t S,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    constexpr int64_t kTile = int64_t(kThreads) * kVec * kMx4Unroll;
    const int lane4 = int(threadIdx.x) & 3;
    for (int64_t base = blockIdx.x * kTile; base < S; base += gridDim.x * kTile) {
        const int64_t i0 = base + int64_t(threadIdx.x) * kVec;
        Group<DT> x[kMx4Unroll];
        if (base + kTile <= S) {
#pragma unroll
            for (int u = 0; u < kMx4Unroll; ++u)
                load_group<DT>(src, i0 + u * (kThreads * kVec), x[u]);
#pragma unroll
            for (int u = 0; u < kMx4Unroll; ++u) {
                const int64_t i = i0 + u * (kThreads * kVec);
                int s;
                const uint32_t w = encode<DT>(x[u], &s);
                __builtin_nontemporal_store(
                    w, reinterpret_cast<g_u32*>(global<g_u8>(codes) + i / 2));
                if (lane4 == 0) global<g_u8>(scales)[i / 32] = uint8_t(s);
            }
        } else {
            // every lane of a quad makes the same trips: they exchange across lanes
#pragma unroll 1
            for (int u = 0; u < kMx4Unroll; ++u) {
                const int64_t i = i0 + u * (kThreads * kVec);
                const int live = i >= S ? 0 : (S - i >= kVec ? kVec : int(S - i));
                load_group_part<DT>(src, i, live, x[0]);
                int s;
                const uint32_t w = encode<DT>(x[0], &s);
                // +0 past the end: the last half byte of an odd shard is 0
#pragma unroll
                for (int k = 0; k < kVec / 2; ++k)
                    if (2 * k < live) global<g_u8>(codes)[i / 2 + k] = uint8_t(w >> (8 * k));
                if (lane4 == 0 && live > 0) global<g_u8>(scales)[i / 32] = uint8_t(s);
            }
        }
    }
}

// Values of a word of codes under scale byte s: 4 words of bf16 pairs or 8 of fp32.
template <int DT>
__device__ __forceinline__ void decode(uint32_t w, int s, Group<DT>& x) {
    if (s != 0 && s != 255) {
        const float two = __uint_as_float(uint32_t(s) << 23);
        if constexpr (DT == ZS_BF16) {
            x.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 0));
            x.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 1));
            x.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 2));
            x.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 3));
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, two, 0);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, two, 1);
            const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, two, 2);
            const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, two, 3);
            const float y[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
            for (int e = 0; e < 8; ++e) x.w[e] = __float_as_uint(y[e]);
        }
    } else {
        float y[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint32_t c = w >> (4 * e);
            y[e] = __builtin_ldexpf(__uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)), s - 1);
            if (s == 255) y[e] = __uint_as_float(0x7fc00000u);
        }
#pragma unroll
        for (int k = 0; k < Group<DT>::words; ++k)
            x.w[k] = DT == ZS_BF16 ? pack_bf16(y[(2 * k) & 7], y[(2 * k + 1) & 7])
                                   : __float_as_uint(y[k & 7]);
    }
}

template <int DT>
__device__ __forceinline__ void store_group(void* dst, int64_t o, const Group<DT>& x) {
    if constexpr (DT == ZS_BF16) {
        __builtin_nontemporal_store(u32x4{x.w[0], x.w[1], x.w[2], x.w[3]},
                                    reinterpret_cast<g_u32x4*>(global<g_u16>(dst) + o));
    } else {
        g_f32* d = global<g_f32>(dst) + o;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            __builtin_nontemporal_store(
                f32x4{__uint_as_float(x.w[4 * k]), __uint_as_float(x.w[4 * k + 1]),
                      __uint_as_float(x.w[4 * k + 2]), __uint_as_float(x.w[4 * k + 3])},
                reinterpret_cast<g_f32x4*>(d + 4 * k));
    }
}

// A unit of 202M bf16 elements from 8 shards: 84 us, 6.1 TB/s (one group a lane and integer
// conversions: 128).
template <int DT>
__global__ __launch_bounds__(kThreads) void gather_mx4_kernel(PtrPack codes, PtrPack scales,
                                                              int64_t S, void* __restrict__ flat) {
    constexpr int64_t kTile = int64_t(kThreads) * kVec * kMx4Unroll;
    const int r = int(blockIdx.y);
    const g_u8* cs = global<const g_u8>(codes.p[r]);
    const g_u8* ss = global<const g_u8>(scales.p[r]);
    const int64_t slot = int64_t(r) * S;
    for (int64_t base = blockIdx.x * kTile; base < S; base += gridDim.x * kTile) {
        const int64_t i0 = base + int64_t(threadIdx.x) * kVec;
        if (base + kTile <= S) {
            uint32_t w[kMx4Unroll];
            int s[kMx4Unroll];
#pragma unroll
            for (int u = 0; u < kMx4Unroll; ++u) {
                const int64_t i = i0 + u * (kThreads * kVec);
                w[u] = __builtin_nontemporal_load(reinterpret_cast<const g_u32*>(cs + i / 2));
                s[u] = ss[i / 32];
            }
#pragma unroll
            for (int u = 0; u < kMx4Unroll; ++u) {
                Group<DT> x;
                decode<DT>(w[u], s[u], x);
                store_group<DT>(flat, slot + i0 + u * (kThreads * kVec), x);
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < kMx4Unroll; ++u) {
                const int64_t i = i0 + u * (kThreads * kVec);
                if (i >= S) break;
                const int live = S - i >= kVec ? kVec : int(S - i);
                uint32_t w = 0;
#pragma unroll
                for (int k = 0; k < kVec / 2; ++k)
                    if (2 * k < live) w |= uint32_t(cs[i / 2 + k]) << (8 * k);
                Group<DT> x;
                decode<DT>(w, ss[i / 32], x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    if (e >= live) continue;
                    if constexpr (DT == ZS_BF16)
                        global<g_u16>(flat)[slot + i + e] =
                            uint16_t(x.w[e / 2] >> (16 * (e & 1)));
                    else
                        global<g_f32>(flat)[slot + i + e] = __uint_as_float(x.w[e]);
                }
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

// Microscaled 4-bit shards for gfx950: quantisation of a bf16 or fp32 shard, and the
// gather that rebuilds a unit from such shards.
//
// Both stream once over their data and are bound by HBM: the quantiser reads 2 or 4
// bytes an element and writes 0.53, the gather reads 0.53 and writes 2 or 4. A lane takes
// 16 bytes of values at a time (8 bf16 or 4 fp32), so that a wavefront's accesses to them
// are one run of 1 KiB, and two such groups, a workgroup apart, whose loads are both ahead
// of their use; 4 or 8 lanes share a block of 32 and its scale byte. (A unit of 202M elements
// gathered to bf16 / fp32: 79 / 149 us; one group 112 / 185, three 82 / 143, four or eight
// 84 / 172, each 7-20% slower or more at odd shard lengths; 8 fp32 values a lane, two stores
// of alternate 16-byte pieces, 330.)
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
constexpr int kBlock = 32;   // elements of a scale byte
constexpr int U = kMx4Groups;  // groups a lane takes of a tile

#define ZS_GLOBAL __attribute__((address_space(1)))
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// vectors at element alignment: a shard, or its slot of the unit, may start at any
// element, and gfx950 accesses it with the same one wide instruction
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_u __attribute__((aligned(1)));
typedef uint16_t u16_u __attribute__((aligned(1)));
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

// A lane's group: 16 bytes of values, E elements, and their codes, one word.
template <int DT>
struct Group;
template <>
struct Group<ZS_BF16> {
    static constexpr int E = 8;
    typedef ZS_GLOBAL u32_u Codes;
    typedef g_u16 Elem;
    uint32_t w[4];  // pairs of elements
};
template <>
struct Group<ZS_F32> {
    static constexpr int E = 4;
    typedef ZS_GLOBAL u16_u Codes;
    typedef g_f32 Elem;
    uint32_t w[4];
};
template <int DT>
constexpr int kTile = kThreads * Group<DT>::E * U;  // elements of a workgroup's tile

// Element i of an array of values.
template <int DT>
__device__ __forceinline__ typename Group<DT>::Elem* value_at(const void* base, int64_t i) {
    return global<typename Group<DT>::Elem>(base) + i;
}
template <int DT>
__device__ __forceinline__ Group<DT> load_group(const void* src, int64_t i) {
    Group<DT> x;
    if constexpr (DT == ZS_BF16) {
        const u32x4 h =
            __builtin_nontemporal_load(reinterpret_cast<const g_u32x4*>(value_at<DT>(src, i)));
#pragma unroll
        for (int k = 0; k < 4; ++k) x.w[k] = h[k];
    } else {
        const f32x4 h =
            __builtin_nontemporal_load(reinterpret_cast<const g_f32x4*>(value_at<DT>(src, i)));
#pragma unroll
        for (int k = 0; k < 4; ++k) x.w[k] = __float_as_uint(h[k]);
    }
    return x;
}
// The first `live` of them, the others +0.
template <int DT>
__device__ __forceinline__ Group<DT> load_group_part(const void* src, int64_t i, int live) {
    Group<DT> x{};
#pragma unroll
    for (int e = 0; e < Group<DT>::E; ++e) {
        if (e >= live) continue;
        if constexpr (DT == ZS_BF16)
            x.w[e / 2] |= uint32_t(*value_at<DT>(src, i + e)) << (16 * (e & 1));
        else
            x.w[e] = __float_as_uint(*value_at<DT>(src, i + e));
    }
    return x;
}
template <int DT>
__device__ __forceinline__ void store_group(void* dst, int64_t i, const Group<DT>& x) {
    if constexpr (DT == ZS_BF16)
        __builtin_nontemporal_store(u32x4{x.w[0], x.w[1], x.w[2], x.w[3]},
                                    reinterpret_cast<g_u32x4*>(value_at<DT>(dst, i)));
    else
        __builtin_nontemporal_store(
            f32x4{__uint_as_float(x.w[0]), __uint_as_float(x.w[1]), __uint_as_float(x.w[2]),
                  __uint_as_float(x.w[3])},
            reinterpret_cast<g_f32x4*>(value_at<DT>(dst, i)));
}
template <int DT>
__device__ __forceinline__ void store_group_part(void* dst, int64_t i, int live,
                                                 const Group<DT>& x) {
#pragma unroll
    for (int e = 0; e < Group<DT>::E; ++e) {
        if (e >= live) continue;
        if constexpr (DT == ZS_BF16)
            *value_at<DT>(dst, i + e) = uint16_t(x.w[e / 2] >> (16 * (e & 1)));
        else
            *value_at<DT>(dst, i + e) = __uint_as_float(x.w[e]);
    }
}
template <int DT>
__device__ __forceinline__ float value_of(const Group<DT>& x, int e) {
    if constexpr (DT == ZS_BF16) return e & 1 ? bf16_hi(x.w[e / 2]) : bf16_lo(x.w[e / 2]);
    else return __uint_as_float(x.w[e]);
}

// The fp32 bits of the largest magnitude of a lane's group (as unsigned numbers: infinity
// and NaN above every number).
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
        for (int k = 0; k < 4; ++k) {
            const uint32_t b = x.w[k] & 0x7fffffffu;
            u = u > b ? u : b;
        }
        return u;
    }
}

// Largest u of the lanes that share a block: 4 with bf16, 8 with fp32.
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t u) {
    const uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(u), CTRL, 0xf, 0xf, true));
    return u > o ? u : o;
}
template <int DT>
__device__ __forceinline__ uint32_t block_max(uint32_t u) {
    u = max_with<0xb1>(u);  // quad_perm 1,0,3,2
    u = max_with<0x4e>(u);  // quad_perm 2,3,0,1
    if constexpr (DT == ZS_F32) u = max_with<0x141>(u);  // row_half_mirror: 7,6,5,4,3,2,1,0
    return u;
}

// Scale byte and codes of a lane's group. Every lane of the block calls it.
template <int DT>
__device__ __forceinline__ uint32_t encode(const Group<DT>& x, int* scale) {
    const uint32_t u = block_max<DT>(top_bits<DT>(x));
    int s = int(u >> 23) - 2;
    s = u >= 0x7f800000u ? 255 : (s > 0 ? s : 0);
    *scale = s;
    uint32_t w = 0;
    if (s != 0 && s != 255) {
        const float two = __uint_as_float(uint32_t(s) << 23);
        if constexpr (DT == ZS_BF16) {
            const auto h = [&](int k) { return __builtin_bit_cast(bf16x2, x.w[k]); };
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, h(0), two, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, h(1), two, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, h(2), two, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, h(3), two, 3);
        } else {
            const auto f = [&](int k) { return __uint_as_float(x.w[k]); };
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(0), f(1), two, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(2), f(3), two, 1);
        }
    } else if (s == 0) {
#pragma unroll
        for (int e = 0; e < Group<DT>::E; ++e) {
            const float y = value_of<DT>(x, e);
            const uint32_t b = __float_as_uint(__builtin_ldexpf(__builtin_fabsf(y), 1 - s));
            uint32_t c = (b + 0x1fffffu + ((b >> 22) & 1u)) >> 22;
            c = c < 7u ? c : 7u;
            w |= (c | ((__float_as_uint(y) >> 31) << 3)) << (4 * e);
        }
    }
    return w;
}

// A bf16 shard of 25.3M elements: 12 us, 5.2 TB/s with the launch's start and end; one of
// 202M 78 us, 6.6 TB/s (fp32 151 us, 6.1), at an odd address 90.
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ src, int64_t S,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    constexpr int E = Group<DT>::E, kStep = kThreads * E;
    const bool first = threadIdx.x % (kBlock / E) == 0;  // of the lanes of a block
    for (int64_t base = blockIdx.x * int64_t(kTile<DT>); base < S;
         base += gridDim.x * int64_t(kTile<DT>)) {
        const int64_t i0 = base + int64_t(threadIdx.x) * E;
        if (base + kTile<DT> <= S) {
            Group<DT> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = load_group<DT>(src, i0 + u * kStep);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * kStep;
                int s;
                typedef typename Group<DT>::Codes C;
                const uint32_t w = encode<DT>(x[u], &s);
                if constexpr (DT == ZS_BF16)
                    __builtin_nontemporal_store(w, reinterpret_cast<C*>(global<g_u8>(codes) + i / 2));
                else
                    *reinterpret_cast<C*>(global<g_u8>(codes) + i / 2) = uint16_t(w);
                if (first) global<g_u8>(scales)[i / kBlock] = uint8_t(s);
            }
        } else {
            // every lane of a block makes the same trips: they exchange across lanes
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * kStep;
                const int live = i >= S ? 0 : (S - i >= E ? E : int(S - i));
                int s;
                const uint32_t w = encode<DT>(load_group_part<DT>(src, i, live), &s);
                // +0 past the end: the last half byte of an odd shard is 0
#pragma unroll
                for (int k = 0; k < E / 2; ++k)
                    if (2 * k < live) global<g_u8>(codes)[i / 2 + k] = uint8_t(w >> (8 * k));
                if (first && live > 0) global<g_u8>(scales)[i / kBlock] = uint8_t(s);
            }
        }
    }
}

// Values of a group's codes under scale byte s.
template <int DT>
__device__ __forceinline__ Group<DT> decode(uint32_t w, int s) {
    Group<DT> x;
    if (s != 0 && s != 255) {
        const float two = __uint_as_float(uint32_t(s) << 23);
        if constexpr (DT == ZS_BF16) {
            const bf16x2 h[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 0),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 1),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 2),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, two, 3)};
#pragma unroll
            for (int k = 0; k < 4; ++k) x.w[k] = __builtin_bit_cast(uint32_t, h[k]);
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, two, 0);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, two, 1);
            x.w[0] = __float_as_uint(a[0]), x.w[1] = __float_as_uint(a[1]);
            x.w[2] = __float_as_uint(b[0]), x.w[3] = __float_as_uint(b[1]);
        }
    } else {
        constexpr int E = Group<DT>::E;
        float y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t c = w >> (4 * e);
            y[e] = __builtin_ldexpf(__uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)), s - 1);
            if (s == 255) y[e] = __uint_as_float(0x7fc00000u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x.w[k] = DT == ZS_BF16 ? pack_bf16(y[(2 * k) % E], y[(2 * k + 1) % E])
                                   : __float_as_uint(y[k % E]);
    }
    return x;
}

// A unit of 202M elements from 8 shards to bf16: 79 us, 6.5 TB/s; from shards of odd length
// 85. To fp32 149 us, 6.2 TB/s.
template <int DT>
__global__ __launch_bounds__(kThreads) void gather_mx4_kernel(PtrPack codes, PtrPack scales,
                                                              int64_t S, void* __restrict__ flat) {
    constexpr int E = Group<DT>::E, kStep = kThreads * E;
    const int r = int(blockIdx.y);
    const g_u8* cs = global<const g_u8>(codes.p[r]);
    const g_u8* ss = global<const g_u8>(scales.p[r]);
    const int64_t slot = int64_t(r) * S;
    for (int64_t base = blockIdx.x * int64_t(kTile<DT>); base < S;
         base += gridDim.x * int64_t(kTile<DT>)) {
        const int64_t i0 = base + int64_t(threadIdx.x) * E;
        if (base + kTile<DT> <= S) {
            uint32_t w[U];
            int s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * kStep;
                typedef const typename Group<DT>::Codes C;
                w[u] = __builtin_nontemporal_load(reinterpret_cast<C*>(cs + i / 2));
                s[u] = ss[i / kBlock];
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                store_group<DT>(flat, slot + i0 + u * kStep, decode<DT>(w[u], s[u]));
        } else {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * kStep;
                if (i >= S) break;
                const int live = S - i >= E ? E : int(S - i);
                uint32_t w = 0;
#pragma unroll
                for (int k = 0; k < E / 2; ++k)
                    if (2 * k < live) w |= uint32_t(cs[i / 2 + k]) << (8 * k);
                store_group_part<DT>(flat, slot + i, live, decode<DT>(w, ss[i / kBlock]));
            }
        }
    }
}

}  // namespace

hipError_t launch_quantize_mx4(const void* src, int dtype, int64_t S, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream) {
    const dim3 grid(unsigned(quantize_mx4_grid(S, dtype == ZS_F32 ? 4 : 2)));
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
    const dim3 grid(unsigned(gather_mx4_grid(S, dtype == ZS_F32 ? 4 : 2, D)), unsigned(D));
    if (dtype == ZS_BF16)
        hipLaunchKernelGGL((gather_mx4_kernel<ZS_BF16>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, flat);
    else
        hipLaunchKernelGGL((gather_mx4_kernel<ZS_F32>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, flat);
    return hipGetLastError();
}

}  // namespace zs

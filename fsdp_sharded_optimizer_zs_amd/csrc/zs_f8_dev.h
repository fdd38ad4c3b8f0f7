// Device code that the kernels of the block-scaled 8-bit matrices share: loads, codes and
// scale bytes of values, values of codes, and stores of a product's elements.
#pragma once

#include "zs_f8.h"
#include "zs_math.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

#define ZS_GLOBAL __attribute__((address_space(1)))
#define ZS_LDS __attribute__((address_space(3)))
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
// vectors at element alignment: a matrix may start at any element of a unit
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef ZS_GLOBAL f32x4_u g_f32x4;
typedef ZS_GLOBAL u32x4_u g_u32x4;
typedef ZS_GLOBAL u32x2_u g_u32x2;
typedef ZS_GLOBAL u32x4 g_u32x4a;
typedef ZS_GLOBAL u32x2 g_u32x2a;
typedef ZS_GLOBAL uint32_t g_u32a;
typedef ZS_GLOBAL uint8_t g_u8;
typedef ZS_GLOBAL uint16_t g_u16;
typedef ZS_GLOBAL float g_f32;

template <typename G, typename P>
__device__ __forceinline__ G* global(P* p) {
    return reinterpret_cast<G*>(reinterpret_cast<uintptr_t>(p));
}

// 8 neighbouring elements of a row.
template <int DT>
struct Eight;
template <>
struct Eight<ZS_BF16> {
    uint32_t w[4];  // pairs
};
template <>
struct Eight<ZS_F32> {
    float f[8];
};

template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void* base, int64_t i) {
    Eight<DT> x;
    if constexpr (DT == ZS_BF16) {
        const u32x4 h = __builtin_nontemporal_load(
            reinterpret_cast<const g_u32x4*>(global<const g_u16>(base) + i));
#pragma unroll
        for (int k = 0; k < 4; ++k) x.w[k] = h[k];
    } else {
        const g_f32x4* p = reinterpret_cast<const g_f32x4*>(global<const g_f32>(base) + i);
        const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) x.f[k] = a[k], x.f[4 + k] = b[k];
    }
    return x;
}
template <int DT>
__device__ __forceinline__ void load1(const void* base, int64_t i, int e, Eight<DT>& x) {
    if constexpr (DT == ZS_BF16)
        x.w[e / 2] |= uint32_t(global<const g_u16>(base)[i]) << (16 * (e & 1));
    else
        x.f[e] = global<const g_f32>(base)[i];
}

// Largest magnitudes as fp32 bits (unsigned numbers: infinity and NaN above every number).
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 mags(uint32_t w) {
    return __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
}
template <int DT>
__device__ __forceinline__ uint32_t top_bits(const Eight<DT>& x) {
    if constexpr (DT == ZS_BF16) {
        u16x2 u = __builtin_elementwise_max(mags(x.w[0]), mags(x.w[1]));
        u = __builtin_elementwise_max(u, __builtin_elementwise_max(mags(x.w[2]), mags(x.w[3])));
        return uint32_t(u[0] > u[1] ? u[0] : u[1]) << 16;
    } else {
        uint32_t u = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) u = max_u(u, __float_as_uint(x.f[k]) & 0x7fffffffu);
        return u;
    }
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t u) {
    return max_u(u, uint32_t(__builtin_amdgcn_mov_dpp(int(u), CTRL, 0xf, 0xf, true)));
}
// Over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row_max(uint32_t u) {
    u = max_with<0xb1>(u);     // quad_perm 1,0,3,2
    u = max_with<0x4e>(u);     // quad_perm 2,3,0,1
    u = max_with<0x141>(u);    // row_half_mirror
    return max_with<0x140>(u); // row_mirror
}
// Over lanes l % 16 = const: gfx950 swaps halves and rows of 16 lanes of two registers, which
// for two copies of one leaves both partners in every lane.
template <typename F>
__device__ __forceinline__ uint32_t over_rows(uint32_t u, F larger) {
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    u = larger(h[0], h[1]);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return larger(r[0], r[1]);
}
__device__ __forceinline__ uint32_t col_max(uint32_t u) {
    return over_rows(u, [](uint32_t a, uint32_t b) { return max_u(a, b); });
}
__device__ __forceinline__ uint32_t col_max_pair(uint32_t u) {  // of the halves apart
    return over_rows(u, [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t,
                                  __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                            __builtin_bit_cast(u16x2, b)));
    });
}

__device__ __forceinline__ int scale_of(uint32_t u, int type) {
    const int s = int((u + 0x1fffffu) >> 23) - (type == ZS_E4M3 ? 8 : 15);
    return u >= 0x7f800000u ? 255 : (s > 1 ? s : 1);
}

// Two codes into half `HI` of a word: gfx950 converts with the scale in one instruction.
// Blocks of s = 1 hold magnitudes that may be subnormal and are scaled by ldexp first.
template <int TYPE, bool HI>
__device__ __forceinline__ uint32_t two_codes(uint32_t w, float a, float b, float two) {
    const s16x2 old = __builtin_bit_cast(s16x2, w);
    if constexpr (TYPE == ZS_E4M3)
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(old, a, b, two, HI));
    else
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(old, a, b, two, HI));
}
template <int TYPE, bool HI>
__device__ __forceinline__ uint32_t two_codes(uint32_t w, uint32_t pair, float two) {
    const s16x2 old = __builtin_bit_cast(s16x2, w);
    const bf16x2 h = __builtin_bit_cast(bf16x2, pair);
    if constexpr (TYPE == ZS_E4M3)
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, h, two, HI));
    else
        return __builtin_bit_cast(uint32_t,
                                  __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(old, h, two, HI));
}

// Whether a block's codes take more than the instruction: it is not finite, or its scale
// byte is 1, where magnitudes may be subnormal (not a block of zeros).
__device__ __forceinline__ bool is_special(uint32_t u, int s) {
    return s == 255 || (s == 1 && u != 0);
}

// 4 codes of values given as pairs of bf16 or as floats, under scale byte s. ANY: also of
// special blocks.
template <int TYPE, bool ANY = true>
__device__ __forceinline__ uint32_t four_codes(float a, float b, float c, float d, int s) {
    float two = __uint_as_float(uint32_t(s) << 23);
    if constexpr (ANY) {
        if (s == 255) return 0;
        if (s == 1) {
            a = __builtin_ldexpf(a, 126), b = __builtin_ldexpf(b, 126);
            c = __builtin_ldexpf(c, 126), d = __builtin_ldexpf(d, 126);
            two = 1.0f;
        }
    }
    return two_codes<TYPE, true>(two_codes<TYPE, false>(0u, a, b, two), c, d, two);
}
template <int TYPE, bool ANY = true>
__device__ __forceinline__ uint32_t four_codes(uint32_t ab, uint32_t cd, int s) {
    if (ANY && (s <= 1 || s == 255))
        return four_codes<TYPE>(bf16_lo(ab), bf16_hi(ab), bf16_lo(cd), bf16_hi(cd), s);
    const float two = __uint_as_float(uint32_t(s) << 23);
    return two_codes<TYPE, true>(two_codes<TYPE, false>(0u, ab, two), cd, two);
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

// Elements [k, k + 8) of row m of p's values x, those past the last column +0.
template <int DT>
__device__ __forceinline__ Eight<DT> eight_of(const F8Product& p, int64_t m, int64_t k) {
    Eight<DT> x{};
    const int64_t at = m * p.ldx + k;
    if (k + 8 <= p.cols) {
        if constexpr (DT == ZS_BF16) {
            const u32x4 h = *reinterpret_cast<const g_u32x4*>(global<const g_u16>(p.x) + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) x.w[e] = h[e];
        } else {
            const g_f32x4* from = reinterpret_cast<const g_f32x4*>(global<const g_f32>(p.x) + at);
            const f32x4 a = from[0], b = from[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) x.f[e] = a[e], x.f[4 + e] = b[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < p.cols) load1<DT>(p.x, at + e, e, x);
    }
    return x;
}

// Codes of 8 elements of a row under scale byte s.
template <int DT, int TYPE, bool ANY = true>
__device__ __forceinline__ u32x2 eight_codes(const Eight<DT>& v, int s) {
    if constexpr (DT == ZS_BF16)
        return u32x2{four_codes<TYPE, ANY>(v.w[0], v.w[1], s),
                     four_codes<TYPE, ANY>(v.w[2], v.w[3], s)};
    else
        return u32x2{four_codes<TYPE, ANY>(v.f[0], v.f[1], v.f[2], v.f[3], s),
                     four_codes<TYPE, ANY>(v.f[4], v.f[5], v.f[6], v.f[7], s)};
}

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

// 16 bytes a lane from base + offset to LDS, lane l's at lds + 16 l. Written as assembly so
// that the compiler's own LDS reads do not wait for it; `arrived` and a barrier do. (The
// instruction takes the LDS address from m0, one wait state after it is written.)
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void load4_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return uint32_t(reinterpret_cast<uintptr_t>((ZS_LDS const void*)(p)));
}

template <int N>
__device__ __forceinline__ void arrived_but() {  // all but the last N loads
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

}  // namespace
}  // namespace zs

// AdamW over many tensors in one launch (moments in fp32 or in 8-bit codes), the
// conversions of the 8-bit moments, and the L2 norm of many gradients, for gfx950.
//
// All are streaming kernels bound by HBM. A workgroup takes one chunk of
// ZS_MULTI_CHUNK elements of one tensor, found in a table in device memory, and
// each of its 4 wavefronts 1024 elements of it, in 4 quarters of 256: lane l holds
// elements 4l .. 4l+3 of each quarter, so that every fp32 access of a wavefront is
// one run of 1 KiB. A quarter is one block of the 8-bit moments, whose scale is
// therefore the same for the whole wavefront: it lives in a scalar register and the
// block's largest magnitude is one reduction over the wavefront.

#include "zs_multi.h"
#include "zs_math.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kThreads = kBlockThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kQ = 4;                      // quarters of a wavefront's elements
constexpr int kQuarter = 256;              // elements of a quarter: a scale block
constexpr int kWaveElems = kQ * kQuarter;  // 1024
static_assert(kWaves * kWaveElems == ZS_MULTI_CHUNK, "a workgroup covers one chunk");

// Tensors start anywhere their elements may (views into a flat unit), so vectors
// are accessed at element alignment: gfx950 does that with the same one wide
// instruction, which costs nothing extra when the address happens to be aligned.
// Pointers read from the table are global memory, never LDS or private memory.
#define ZS_GLOBAL __attribute__((address_space(1)))
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_u __attribute__((aligned(1)));
typedef ZS_GLOBAL f32x4_u g_f32x4;
typedef ZS_GLOBAL u32x2_u g_u32x2;
typedef ZS_GLOBAL u32_u g_u32;
typedef ZS_GLOBAL float g_f32;
typedef ZS_GLOBAL uint16_t g_u16;
typedef ZS_GLOBAL uint8_t g_u8;

template <typename G, typename P>
__device__ __forceinline__ G* global(P* p) {
    return reinterpret_cast<G*>(reinterpret_cast<uintptr_t>(p));
}

// Four consecutive gradient elements, widened: whole (lanes of a full quarter)
// or the first `live` of them, the others 0.
template <int DT>
__device__ __forceinline__ void load_grad(const void* base, int64_t i, float (&x)[4]) {
    if constexpr (DT == ZS_BF16) {
        const u32x2 h = __builtin_nontemporal_load(
            reinterpret_cast<const g_u32x2*>(global<const g_u16>(base) + i));
        x[0] = bf16_lo(h[0]), x[1] = bf16_hi(h[0]), x[2] = bf16_lo(h[1]), x[3] = bf16_hi(h[1]);
    } else {
        const f32x4 a = __builtin_nontemporal_load(
            reinterpret_cast<const g_f32x4*>(global<const g_f32>(base) + i));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a[e];
    }
}
template <int DT>
__device__ __forceinline__ void load_grad_part(const void* base, int64_t i, int live,
                                               float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = 0.0f;
        if (e < live) {
            if constexpr (DT == ZS_BF16)
                x[e] = __uint_as_float(uint32_t(global<const g_u16>(base)[i + e]) << 16);
            else
                x[e] = global<const g_f32>(base)[i + e];
        }
    }
}

__device__ __forceinline__ void load_f32(const float* base, int64_t i, float (&x)[4]) {
    const f32x4 a = __builtin_nontemporal_load(
        reinterpret_cast<const g_f32x4*>(global<const g_f32>(base) + i));
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a[e];
}
__device__ __forceinline__ void load_f32_part(const float* base, int64_t i, int live,
                                              float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = e < live ? global<const g_f32>(base)[i + e] : 0.0f;
}
__device__ __forceinline__ void store_f32(float* base, int64_t i, const float (&x)[4]) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]},
                                reinterpret_cast<g_f32x4*>(global<g_f32>(base) + i));
}
__device__ __forceinline__ void store_f32_part(float* base, int64_t i, int live,
                                               const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) global<g_f32>(base)[i + e] = x[e];
}
__device__ __forceinline__ void store_bf16(uint16_t* base, int64_t i, const float (&x)[4]) {
    const u32x2 h{f32_to_bf16(x[0]) | (f32_to_bf16(x[1]) << 16),
                  f32_to_bf16(x[2]) | (f32_to_bf16(x[3]) << 16)};
    __builtin_nontemporal_store(h, reinterpret_cast<g_u32x2*>(global<g_u16>(base) + i));
}
__device__ __forceinline__ void store_bf16_part(uint16_t* base, int64_t i, int live,
                                                const float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) global<g_u16>(base)[i + e] = uint16_t(f32_to_bf16(x[e]));
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t* base, int64_t i) {
    return __builtin_nontemporal_load(
        reinterpret_cast<const g_u32*>(global<const g_u8>(base) + i));
}
__device__ __forceinline__ uint32_t load_codes_part(const uint8_t* base, int64_t i, int live) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) w |= uint32_t(global<const g_u8>(base)[i + e]) << (8 * e);
    return w;
}
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t i, uint32_t w) {
    __builtin_nontemporal_store(w, reinterpret_cast<g_u32*>(global<g_u8>(base) + i));
}
__device__ __forceinline__ void store_codes_part(uint8_t* base, int64_t i, int live, uint32_t w) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) global<g_u8>(base)[i + e] = uint8_t(w >> (8 * e));
}

// Elements of [i, n) that a lane's four hold: 0 .. 4.
__device__ __forceinline__ int live_of(int64_t i, int64_t n) {
    return i >= n ? 0 : (n - i >= 4 ? 4 : int(n - i));
}

// ------------------------------------------------------------- 8-bit moments

// A code is the top of an fp32 pattern: 3 bits of mantissa and 4 (m, plus a sign)
// or 5 (v) of exponent, so that widening is a shift and fp32's own subnormals are
// the code's, and 2^(s - K) puts it in its block's range (K: the top code's
// exponent field).
template <bool SIGNED>
struct Code;
template <>
struct Code<true> {
    static constexpr int K = 15, most = 127, least_scale = 0;
};
template <>
struct Code<false> {
    static constexpr int K = 31, most = 255, least_scale = 11;
};

// Values of four codes under scale byte s (the same for the wavefront).
template <bool SIGNED>
__device__ __forceinline__ void decode4(uint32_t w, int s, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t c = (w >> (8 * e)) & 0xffu;
        const uint32_t bits = SIGNED ? ((c & 0x7fu) << 20) | ((c & 0x80u) << 24) : c << 20;
        x[e] = __builtin_ldexpf(__uint_as_float(bits), s - Code<SIGNED>::K);
    }
    if (s == 255) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(0x7fc00000u);
    }
}

// The scale byte of a block whose largest magnitude has the bits u.
template <bool SIGNED>
__device__ __forceinline__ int scale_of(uint32_t u) {
    if (u >= 0x7f800000u) return 255;
    int s = int((u + 0xfffffu) >> 23);
    s = s < 254 ? s : 254;
    return s > Code<SIGNED>::least_scale ? s : Code<SIGNED>::least_scale;
}

// Codes of four values under scale byte s; rnd[e]: the element's 16 random bits
// (STOCH) in the low half.
template <bool SIGNED, bool STOCH>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], int s, const uint32_t (&rnd)[4]) {
    uint32_t w = 0;
    if (s == 255) return w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t b =
            __float_as_uint(__builtin_ldexpf(__builtin_fabsf(x[e]), Code<SIGNED>::K - s));
        const uint32_t add = STOCH ? ((rnd[e] & 0xffffu) << 4) | 8u : 0x7ffffu + ((b >> 20) & 1u);
        uint32_t c = (b + add) >> 20;
        c = c < uint32_t(Code<SIGNED>::most) ? c : uint32_t(Code<SIGNED>::most);
        if constexpr (SIGNED) {
            c |= (__float_as_uint(x[e]) >> 31) << 7;
        } else {
            c = x[e] > 0.0f ? (c > 1u ? c : 1u) : 0u;
        }
        w |= c << (8 * e);
    }
    return w;
}

// Largest of the wavefront's u (as unsigned numbers: a NaN's bits are above
// infinity's, infinity's above every number's), in a scalar register. The row
// rotations of DPP reduce each row of 16 lanes; the 4 rows' values are read out.
template <int CTRL>
__device__ __forceinline__ uint32_t max_row(uint32_t u) {
    const uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(u), CTRL, 0xf, 0xf, true));
    return u > o ? u : o;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t u) {
    u = max_row<0x121>(u);  // row_ror:1
    u = max_row<0x122>(u);  // row_ror:2
    u = max_row<0x124>(u);  // row_ror:4
    u = max_row<0x128>(u);  // row_ror:8
    const uint32_t a = uint32_t(__builtin_amdgcn_readlane(int(u), 0));
    const uint32_t b = uint32_t(__builtin_amdgcn_readlane(int(u), 16));
    const uint32_t c = uint32_t(__builtin_amdgcn_readlane(int(u), 32));
    const uint32_t d = uint32_t(__builtin_amdgcn_readlane(int(u), 48));
    const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
    return ab > cd ? ab : cd;
}
__device__ __forceinline__ uint32_t top_bits(const float (&x)[4]) {
    uint32_t u = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t b = __float_as_uint(x[e]) & 0x7fffffffu;
        u = u > b ? u : b;
    }
    return u;
}

__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x *= 0x6a09e667u;
    x ^= x >> 15;
    x *= 0xbb67ae85u;
    return x ^ (x >> 16);
}

// ------------------------------------------------------------- the step

// fp32 moments: one quarter, whole or the first `live` elements of each lane.
template <int DT, bool FULL>
__device__ __forceinline__ void step32(const zs_multi_tensor& t, int64_t i, int live,
                                       const MultiArgs& a, float mult) {
    float p[4], m[4], v[4], g[4];
    if constexpr (FULL) {
        load_f32(t.p, i, p);
        load_f32(static_cast<const float*>(t.m), i, m);
        load_f32(static_cast<const float*>(t.v), i, v);
        load_grad<DT>(t.g, i, g);
    } else {
        load_f32_part(t.p, i, live, p);
        load_f32_part(static_cast<const float*>(t.m), i, live, m);
        load_f32_part(static_cast<const float*>(t.v), i, live, v);
        load_grad_part<DT>(t.g, i, live, g);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) adamw1(p[e], m[e], v[e], g[e] * mult, a.k);
    if constexpr (FULL) {
        store_f32(t.p, i, p);
        store_f32(static_cast<float*>(t.m), i, m);
        store_f32(static_cast<float*>(t.v), i, v);
        if (t.w_out) store_bf16(t.w_out, i, p);
    } else {
        store_f32_part(t.p, i, live, p);
        store_f32_part(static_cast<float*>(t.m), i, live, m);
        store_f32_part(static_cast<float*>(t.v), i, live, v);
        if (t.w_out) store_bf16_part(t.w_out, i, live, p);
    }
}

// 8-bit moments: the same, the quarter's scale bytes sm and sv in and out.
template <int DT, bool STOCH, bool FULL>
__device__ __forceinline__ void step8(const zs_multi_tensor& t, int64_t i, int live,
                                      const MultiArgs& a, float mult, uint32_t key, int* sm,
                                      int* sv) {
    float p[4], m[4], v[4], g[4];
    uint8_t* const mc = static_cast<uint8_t*>(t.m);
    uint8_t* const vc = static_cast<uint8_t*>(t.v);
    uint32_t wm, wv;
    if constexpr (FULL) {
        load_f32(t.p, i, p);
        wm = load_codes(mc, i);
        wv = load_codes(vc, i);
        load_grad<DT>(t.g, i, g);
    } else {
        load_f32_part(t.p, i, live, p);
        wm = load_codes_part(mc, i, live);
        wv = load_codes_part(vc, i, live);
        load_grad_part<DT>(t.g, i, live, g);
    }
    decode4<true>(wm, *sm, m);
    decode4<false>(wv, *sv, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        adamw1(p[e], m[e], v[e], g[e] * mult, a.k);
        if (!FULL && e >= live) m[e] = v[e] = 0.0f;  // no part of the block's largest
    }
    *sm = scale_of<true>(wave_max(top_bits(m)));
    *sv = scale_of<false>(wave_max(top_bits(v)));
    uint32_t rm[4] = {}, rv[4] = {};
    if constexpr (STOCH) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t r = mix(uint32_t(i + e) ^ key);
            rm[e] = r;
            rv[e] = r >> 16;
        }
    }
    wm = encode4<true, STOCH>(m, *sm, rm);
    wv = encode4<false, STOCH>(v, *sv, rv);
    if constexpr (FULL) {
        store_f32(t.p, i, p);
        if (t.w_out) store_bf16(t.w_out, i, p);
        store_codes(mc, i, wm);
        store_codes(vc, i, wv);
    } else {
        store_f32_part(t.p, i, live, p);
        if (t.w_out) store_bf16_part(t.w_out, i, live, p);
        store_codes_part(mc, i, live, wm);
        store_codes_part(vc, i, live, wv);
    }
}

template <int DT, int STATE, bool STOCH>
__global__ __launch_bounds__(kThreads) void multi_kernel(
    const zs_multi_tensor* __restrict__ table, const MultiChunk* __restrict__ chunks,
    int64_t n_chunks, MultiArgs a) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const float mult = a.grad_scale ? *a.grad_scale : 1.0f;
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const MultiChunk ch = chunks[c];
        const zs_multi_tensor t = table[ch.tensor];
        const int64_t n = t.numel;
        const int64_t base = int64_t(ch.index) * ZS_MULTI_CHUNK + wave * kWaveElems;
        if (base >= n) continue;
        if constexpr (STATE == ZS_STATE_F32) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const int64_t i = base + q * kQuarter + 4 * lane;
                if (base + (q + 1) * kQuarter <= n) {
                    step32<DT, true>(t, i, 4, a, mult);
                } else if (base + q * kQuarter < n) {
                    step32<DT, false>(t, i, live_of(i, n), a, mult);
                }
            }
        } else {
            const uint32_t key = STOCH ? mix(mix(a.seed_lo + 0x9e3779b9u * uint32_t(ch.tensor + 1)) +
                                             a.seed_hi)
                                       : 0u;
            // lane q holds the scale bytes of quarter q
            const int64_t block0 = base / kQuarter;
            const bool mine = lane < kQ && base + lane * kQuarter < n;
            int lm = 0, lv = 0;
            if (mine) {
                lm = global<const g_u8>(t.m_scale)[block0 + lane];
                lv = global<const g_u8>(t.v_scale)[block0 + lane];
            }
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const int64_t i = base + q * kQuarter + 4 * lane;
                if (base + q * kQuarter >= n) break;
                int sm = __builtin_amdgcn_readlane(lm, q);
                int sv = __builtin_amdgcn_readlane(lv, q);
                if (base + (q + 1) * kQuarter <= n)
                    step8<DT, STOCH, true>(t, i, 4, a, mult, key, &sm, &sv);
                else
                    step8<DT, STOCH, false>(t, i, live_of(i, n), a, mult, key, &sm, &sv);
                if (lane == q) {
                    lm = sm;
                    lv = sv;
                }
            }
            if (mine) {
                global<g_u8>(t.m_scale)[block0 + lane] = uint8_t(lm);
                global<g_u8>(t.v_scale)[block0 + lane] = uint8_t(lv);
            }
        }
    }
}

// ------------------------------------------------------------- conversions

// One block of 256 elements per wavefront.
template <bool SIGNED>
__global__ __launch_bounds__(kThreads) void encode8_kernel(const float* __restrict__ x, int64_t S,
                                                           uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int64_t blocks = (S + kQuarter - 1) / kQuarter;
    const uint32_t none[4] = {};
    for (int64_t b = int64_t(blockIdx.x) * kWaves + wave; b < blocks;
         b += int64_t(gridDim.x) * kWaves) {
        const int64_t i = b * kQuarter + 4 * lane;
        const int live = live_of(i, S);
        float y[4];
        if (live == 4) load_f32(x, i, y);
        else load_f32_part(x, i, live, y);
        if constexpr (!SIGNED) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (y[e] < 0.0f) y[e] = __uint_as_float(0x7fc00000u);
        }
        const int s = scale_of<SIGNED>(wave_max(top_bits(y)));
        const uint32_t w = encode4<SIGNED, false>(y, s, none);
        if (live == 4) store_codes(codes, i, w);
        else store_codes_part(codes, i, live, w);
        if (lane == 0) global<g_u8>(scales)[b] = uint8_t(s);
    }
}

template <bool SIGNED, int DT>
__global__ __launch_bounds__(kThreads) void decode8_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           int64_t S, void* __restrict__ out) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int64_t blocks = (S + kQuarter - 1) / kQuarter;
    for (int64_t b = int64_t(blockIdx.x) * kWaves + wave; b < blocks;
         b += int64_t(gridDim.x) * kWaves) {
        const int64_t i = b * kQuarter + 4 * lane;
        const int live = live_of(i, S);
        const int s = __builtin_amdgcn_readfirstlane(int(global<const g_u8>(scales)[b]));
        const uint32_t w = live == 4 ? load_codes(codes, i) : load_codes_part(codes, i, live);
        float x[4];
        decode4<SIGNED>(w, s, x);
        if constexpr (DT == ZS_F32) {
            if (live == 4) store_f32(static_cast<float*>(out), i, x);
            else store_f32_part(static_cast<float*>(out), i, live, x);
        } else {
            if (live == 4) store_bf16(static_cast<uint16_t*>(out), i, x);
            else store_bf16_part(static_cast<uint16_t*>(out), i, live, x);
        }
    }
}

// ------------------------------------------------------------- the norm

// Sum over the workgroup, in a fixed order, valid in thread 0.
__device__ __forceinline__ double block_sum(double x, double* slot) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += slot[w];
    }
    return s;
}

// Partial sums of squares: workgroup b takes chunks b, b + gridDim.x, ... In fp64,
// where the product of two fp32 numbers is exact and no square over- or underflows.
template <int DT>
__global__ __launch_bounds__(kThreads) void sumsq_kernel(const zs_multi_tensor* __restrict__ table,
                                                         const MultiChunk* __restrict__ chunks,
                                                         int64_t n_chunks,
                                                         double* __restrict__ partial) {
    __shared__ double slot[kWaves];
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const MultiChunk ch = chunks[c];
        const void* g = table[ch.tensor].g;
        const int64_t n = table[ch.tensor].numel;
        const int64_t base = int64_t(ch.index) * ZS_MULTI_CHUNK + wave * kWaveElems;
        float x[kQ][4];
        if (base + kWaveElems <= n) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) load_grad<DT>(g, base + q * kQuarter + 4 * lane, x[q]);
        } else {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const int64_t i = base + q * kQuarter + 4 * lane;
                load_grad_part<DT>(g, i, live_of(i, n), x[q]);
            }
        }
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = __builtin_fma(double(x[q][e]), double(x[q][e]), s[e]);
    }
    const double t = block_sum((s[0] + s[1]) + (s[2] + s[3]), slot);
    if (threadIdx.x == 0) partial[blockIdx.x] = t;
}

__device__ __forceinline__ void write_clip(double sum, double max_norm, float* norm_coef) {
    const double norm = __builtin_sqrt(sum);
    norm_coef[0] = float(norm);
    float c = 1.0f;
    if (!__builtin_isinf(max_norm)) {
        const double d = max_norm / (norm + 1e-6);
        c = d >= 1.0 ? 1.0f : float(d);
    }
    norm_coef[1] = c;
}

__global__ __launch_bounds__(kThreads) void norm_final_kernel(const double* __restrict__ partial,
                                                              int n, double max_norm,
                                                              double* __restrict__ sumsq,
                                                              float* __restrict__ norm_coef) {
    __shared__ double slot[kWaves];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
    s = block_sum(s, slot);
    if (threadIdx.x == 0) {
        *sumsq = s;
        write_clip(s, max_norm, norm_coef);
    }
}

__global__ __launch_bounds__(64) void clip_kernel(PtrPack sums, int D, double max_norm,
                                                  float* __restrict__ norm_coef) {
    if (threadIdx.x != 0) return;
    double s = 0.0;
    for (int r = 0; r < D; ++r) s += *static_cast<const double*>(sums.p[r]);
    write_clip(s, max_norm, norm_coef);
}

template <int DT, int STATE, bool STOCH>
hipError_t launch_kind(const MultiImage& im, const MultiArgs& a, hipStream_t stream) {
    const unsigned grid = unsigned(grid_blocks(im.n_chunks, 1));
    hipLaunchKernelGGL((multi_kernel<DT, STATE, STOCH>), dim3(grid), dim3(kThreads), 0, stream,
                       im.table, im.chunks, im.n_chunks, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_multi(const MultiImage& im, int state, int dtype, const MultiArgs& a, bool stoch,
                        hipStream_t stream) {
    if (state == ZS_STATE_F32) {
        return dtype == ZS_BF16 ? launch_kind<ZS_BF16, ZS_STATE_F32, false>(im, a, stream)
                                : launch_kind<ZS_F32, ZS_STATE_F32, false>(im, a, stream);
    }
    if (stoch) {
        return dtype == ZS_BF16 ? launch_kind<ZS_BF16, ZS_STATE_8BIT, true>(im, a, stream)
                                : launch_kind<ZS_F32, ZS_STATE_8BIT, true>(im, a, stream);
    }
    return dtype == ZS_BF16 ? launch_kind<ZS_BF16, ZS_STATE_8BIT, false>(im, a, stream)
                            : launch_kind<ZS_F32, ZS_STATE_8BIT, false>(im, a, stream);
}

hipError_t launch_encode8(const float* x, int64_t S, bool is_signed, uint8_t* codes,
                          uint8_t* scales, hipStream_t stream) {
    const dim3 grid(unsigned(state8_grid(S)));
    if (is_signed)
        hipLaunchKernelGGL((encode8_kernel<true>), grid, dim3(kThreads), 0, stream, x, S, codes,
                           scales);
    else
        hipLaunchKernelGGL((encode8_kernel<false>), grid, dim3(kThreads), 0, stream, x, S, codes,
                           scales);
    return hipGetLastError();
}

hipError_t launch_decode8(const uint8_t* codes, const uint8_t* scales, int64_t S, bool is_signed,
                          int dtype, void* out, hipStream_t stream) {
    const dim3 grid(unsigned(state8_grid(S)));
    if (is_signed && dtype == ZS_F32)
        hipLaunchKernelGGL((decode8_kernel<true, ZS_F32>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, out);
    else if (is_signed)
        hipLaunchKernelGGL((decode8_kernel<true, ZS_BF16>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, out);
    else if (dtype == ZS_F32)
        hipLaunchKernelGGL((decode8_kernel<false, ZS_F32>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, out);
    else
        hipLaunchKernelGGL((decode8_kernel<false, ZS_BF16>), grid, dim3(kThreads), 0, stream, codes,
                           scales, S, out);
    return hipGetLastError();
}

hipError_t launch_norm(const MultiImage& im, int dtype, double max_norm, double* sumsq,
                       float* norm_coef, double* partial, hipStream_t stream) {
    const int n = int(norm_grid(im.n_chunks));
    if (n > 0) {
        if (dtype == ZS_BF16)
            hipLaunchKernelGGL((sumsq_kernel<ZS_BF16>), dim3(unsigned(n)), dim3(kThreads), 0,
                               stream, im.table, im.chunks, im.n_chunks, partial);
        else
            hipLaunchKernelGGL((sumsq_kernel<ZS_F32>), dim3(unsigned(n)), dim3(kThreads), 0, stream,
                               im.table, im.chunks, im.n_chunks, partial);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(norm_final_kernel, dim3(1), dim3(kThreads), 0, stream, partial, n, max_norm,
                       sumsq, norm_coef);
    return hipGetLastError();
}

hipError_t launch_clip(const PtrPack& sums, int D, double max_norm, float* norm_coef,
                       hipStream_t stream) {
    hipLaunchKernelGGL(clip_kernel, dim3(1), dim3(64), 0, stream, sums, D, max_norm, norm_coef);
    return hipGetLastError();
}

}  // namespace zs

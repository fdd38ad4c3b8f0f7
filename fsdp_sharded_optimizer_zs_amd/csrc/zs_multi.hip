// AdamW over many tensors in one launch (moments in fp32 or in 8-bit codes), the
// conversions of the 8-bit moments, and the L2 norm of many gradients, for gfx950.
//
// All are streaming kernels bound by HBM. A workgroup takes one chunk of at most
// ZS_MULTI_CHUNK elements of one tensor, described in device memory, and each of its 4
// wavefronts 1024 elements of it, in 4 quarters of 256: lane l holds elements 4l .. 4l+3
// of each quarter, so that every fp32 access of a wavefront is one run of 1 KiB. A quarter
// is one block of the 8-bit moments, whose scale is therefore the same for the whole
// wavefront: it lives in a scalar register and the block's largest magnitude is one
// reduction over the wavefront.

#include "zs_multi.h"
#include "zs_math.h"
#include "zs_norm.h"

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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_u __attribute__((aligned(1)));
typedef ZS_GLOBAL f32x4_u g_f32x4;
typedef ZS_GLOBAL u32x2_u g_u32x2;
typedef ZS_GLOBAL u32_u g_u32;
typedef ZS_GLOBAL float g_f32;
typedef ZS_GLOBAL uint16_t g_u16;
typedef ZS_GLOBAL uint8_t g_u8;

// Element q * kQuarter + i of an array whose base scalar registers hold: i is the lane's
// own 32-bit offset and the quarter's goes into the instruction.
template <typename G>
__device__ __forceinline__ G* element(const void* base, int q, uint32_t i) {
    return reinterpret_cast<G*>(reinterpret_cast<uintptr_t>(base) +
                                uint32_t(q) * uint32_t(kQuarter * sizeof(G)) +
                                i * uint32_t(sizeof(G)));
}

// Elements of [i, n) that a lane's four hold: 0 .. 4.
__device__ __forceinline__ int live_of(int i, int n) {
    return i >= n ? 0 : (n - i >= 4 ? 4 : n - i);
}

// A lane's four elements of quarter q, from its i on, of which the first `live` exist (the
// others read as 0 and are not written). Lanes whose four all exist access them at once;
// with ALL every lane does, and `live` is not looked at. Streams are touched once a step
// and go by non-temporal accesses, except (CACHED) where a whole step stays in the
// memory-side cache until the next one.
template <bool ALL, bool CACHED = false>
__device__ __forceinline__ void load_f32(const float* base, int q, uint32_t i, int live,
                                         float (&x)[4]) {
    const g_f32* s = element<const g_f32>(base, q, i);
    if (ALL || live == 4) {
        const g_f32x4* v = reinterpret_cast<const g_f32x4*>(s);
        const f32x4 a = CACHED ? f32x4(*v) : f32x4(__builtin_nontemporal_load(v));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = e < live ? s[e] : 0.0f;
    }
}
template <bool ALL, bool CACHED = false>
__device__ __forceinline__ void store_f32(float* base, int q, uint32_t i, int live,
                                          const float (&x)[4]) {
    g_f32* d = element<g_f32>(base, q, i);
    if (ALL || live == 4) {
        g_f32x4* v = reinterpret_cast<g_f32x4*>(d);
        const f32x4 a{x[0], x[1], x[2], x[3]};
        if constexpr (CACHED) *v = a;
        else __builtin_nontemporal_store(a, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < live) d[e] = x[e];
    }
}
// Gradients, widened.
template <int DT, bool ALL, bool CACHED = false>
__device__ __forceinline__ void load_grad(const void* base, int q, uint32_t i, int live,
                                          float (&x)[4]) {
    if constexpr (DT == ZS_F32) {
        load_f32<ALL, CACHED>(static_cast<const float*>(base), q, i, live, x);
    } else {
        const g_u16* s = element<const g_u16>(base, q, i);
        u32x2 h{0, 0};
        if (ALL || live == 4) {
            const g_u32x2* v = reinterpret_cast<const g_u32x2*>(s);
            h = CACHED ? u32x2(*v) : u32x2(__builtin_nontemporal_load(v));
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < live) h[e / 2] |= uint32_t(s[e]) << (16 * (e & 1));
        }
        x[0] = bf16_lo(h[0]), x[1] = bf16_hi(h[0]), x[2] = bf16_lo(h[1]), x[3] = bf16_hi(h[1]);
    }
}
template <bool ALL, bool CACHED = false>
__device__ __forceinline__ void store_bf16(uint16_t* base, int q, uint32_t i, int live,
                                           const float (&x)[4]) {
    g_u16* d = element<g_u16>(base, q, i);
    const u32x2 h{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    if (ALL || live == 4) {
        g_u32x2* v = reinterpret_cast<g_u32x2*>(d);
        if constexpr (CACHED) *v = h;
        else __builtin_nontemporal_store(h, v);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < live) d[e] = uint16_t(h[e / 2] >> (16 * (e & 1)));
    }
}
template <bool ALL>
__device__ __forceinline__ uint32_t load_codes(const void* base, int q, uint32_t i, int live) {
    const g_u8* s = element<const g_u8>(base, q, i);
    uint32_t w = 0;
    if (ALL || live == 4) {
        w = __builtin_nontemporal_load(reinterpret_cast<const g_u32*>(s));
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < live) w |= uint32_t(s[e]) << (8 * e);
    }
    return w;
}
template <bool ALL>
__device__ __forceinline__ void store_codes(void* base, int q, uint32_t i, int live, uint32_t w) {
    g_u8* d = element<g_u8>(base, q, i);
    if (ALL || live == 4) {
        __builtin_nontemporal_store(w, reinterpret_cast<g_u32*>(d));
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < live) d[e] = uint8_t(w >> (8 * e));
    }
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

// fp32 moments: a wavefront's 1024 elements, those below n (i: the lane's first); every
// load ahead of the arithmetic, and each quarter stored as soon as it is done.
// Bound by HBM: 202M parameters with bf16 gradients 940 us, 6.0 TB/s, where a copy reaches
// 6.57. In one process, at 931: storing stream by stream after all four quarters 993,
// loading two quarters at a time 951, one at a time 954, fewer wavefronts a SIMD 944-965,
// temporal loads 1019; at 945: six or eight wavefronts a SIMD 959 and 1029.
template <int DT, bool ALL, bool CACHED>
__device__ __forceinline__ void step32_wave(const MultiChunk& t, int i, int n,
                                            const MultiArgs& a, float mult) {
    float* const tm = static_cast<float*>(t.m);
    float* const tv = static_cast<float*>(t.v);
    float p[kQ][4], m[kQ][4], v[kQ][4], g[kQ][4];
    int live[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        live[q] = ALL ? 4 : live_of(q * kQuarter + i, n);
        load_f32<ALL, CACHED>(t.p, q, i, live[q], p[q]);
        load_f32<ALL, CACHED>(tm, q, i, live[q], m[q]);
        load_f32<ALL, CACHED>(tv, q, i, live[q], v[q]);
        load_grad<DT, ALL, CACHED>(t.g, q, i, live[q], g[q]);
    }
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) adamw1(p[q][e], m[q][e], v[q][e], g[q][e] * mult, a.k);
        store_f32<ALL, CACHED>(t.p, q, i, live[q], p[q]);
        store_f32<ALL, CACHED>(tm, q, i, live[q], m[q]);
        store_f32<ALL, CACHED>(tv, q, i, live[q], v[q]);
        if (t.w_out) store_bf16<ALL, CACHED>(t.w_out, q, i, live[q], p[q]);
    }
}

// The parameter's part of the update with 8-bit moments. EXACT: the fp32 step's
// operations, each correctly rounded. Otherwise the root and the two quotients are
// the hardware's one-step approximations and a product with 1 / BC2S: 10 issue slots
// instead of about 50, of which HBM leaves about 100 an element. Their errors (root and
// reciprocal one ulp, 1 / BC2S, divisor and product half of one: 7 * 2^-24) stay within
// 2^-21 of the update, but for an m' / den in the subnormals, which is off by 2^-150 as in
// the fp32 step. It needs EPS * BC2S >= 2^-38: then the roots that the hardware may flush (of
// subnormals, so at most 2^-63 / BC2S of the divisor) are below half an ulp of EPS. And it
// needs EPS <= 2^125: the hardware gives 0 for a subnormal reciprocal, and beside EPS the
// divisor has at most 2^64 / BC2S < 2^91, so that it stays below 2^126.
template <bool EXACT>
__device__ __forceinline__ float new_p(float p, float m1, float v1, const MultiArgs& a) {
    if constexpr (EXACT) {
        const float den = (__builtin_sqrtf(v1) / a.k.bc2s) + a.k.eps;
        return (p * a.k.dec) - (a.k.ss * (m1 / den));
    } else {
        const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v1), a.rbc2s, a.k.eps);
        return __builtin_fmaf(-a.k.ss, m1 * __builtin_amdgcn_rcpf(den), p * a.k.dec);
    }
}

__device__ __forceinline__ uint32_t tensor_key(const MultiArgs& a, int32_t tensor) {
    return mix(mix(a.seed_lo + 0x9e3779b9u * uint32_t(tensor + 1)) + a.seed_hi);
}

// 8-bit moments, any case: one quarter, the first `live` elements of each lane, its
// scale bytes sm and sv in and out.
template <int DT, bool STOCH, bool EXACT>
__device__ __forceinline__ void step8_quarter(const MultiChunk& t, int q, int i, int live,
                                              const MultiArgs& a, float mult, uint32_t key,
                                              int* sm, int* sv) {
    float p[4], m[4], v[4], g[4];
    load_f32<false>(t.p, q, i, live, p);
    load_grad<DT, false>(t.g, q, i, live, g);
    decode4<true>(load_codes<false>(t.m, q, i, live), *sm, m);
    decode4<false>(load_codes<false>(t.v, q, i, live), *sv, v);
    uint32_t rm[4] = {}, rv[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = g[e] * mult;
        m[e] = (a.k.b1 * m[e]) + (a.k.b1c * x);
        v[e] = (a.k.b2 * v[e]) + (a.k.b2c * (x * x));
        p[e] = new_p<EXACT>(p[e], m[e], v[e], a);
        if (e >= live) m[e] = v[e] = 0.0f;  // no part of the block's largest
        if constexpr (STOCH) {
            rm[e] = mix((t.first + uint32_t(q * kQuarter + i + e)) ^ key);
            rv[e] = rm[e] >> 16;
        }
    }
    *sm = scale_of<true>(wave_max(top_bits(m)));
    *sv = scale_of<false>(wave_max(top_bits(v)));
    store_codes<false>(t.m, q, i, live, encode4<true, STOCH>(m, *sm, rm));
    store_codes<false>(t.v, q, i, live, encode4<false, STOCH>(v, *sv, rv));
    store_f32<false>(t.p, q, i, live, p);
    if (t.w_out) store_bf16<false>(t.w_out, q, i, live, p);
}

// Codes as encode4 gives them, for a scale byte below 254: then the largest magnitude
// is at most the top code's value and no code needs a limit. Signs ride along in bit
// 31 (the sum never reaches it); the codes are packed from whole bytes.
template <bool STOCH>
__device__ __forceinline__ uint32_t pack_m(const float (&x)[4], int s, const uint32_t (&r)[4]) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t u = __float_as_uint(__builtin_ldexpf(x[e], Code<true>::K - s));
        u += STOCH ? ((r[e] << 4) & 0xffff0u) | 8u : 0x7ffffu + ((u >> 20) & 1u);
        c[e] = ((u << 4) & 0x7fffffffu) | (u & 0x80000000u);
    }
    return __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0703u) |
           __builtin_amdgcn_perm(c[3], c[2], 0x07030c0cu);
}
template <bool STOCH>
__device__ __forceinline__ uint32_t pack_v(const float (&x)[4], int s, const uint32_t (&r)[4]) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t u = __float_as_uint(__builtin_ldexpf(x[e], Code<false>::K - s));
        u += STOCH ? ((r[e] >> 12) & 0xffff0u) | 8u : 0x7ffffu + ((u >> 20) & 1u);
        const uint32_t b = __float_as_uint(x[e]), one = b < 1u ? b : 1u;  // 1 for x > 0
        const uint32_t k = u >> 20;
        c[e] = k > one ? k : one;
    }
    return __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u) |
           __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
}

// Order the wavefront's LDS accesses before and after this point.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// HBM is written in 64-byte sectors, and one that two store instructions share is written
// twice. The blocks of the 8-bit moments fix which elements a wavefront has, so that p and
// w_out of a tensor off the sectors would share one between every two quarters. Their new
// values go through the wavefront's slot of LDS instead and leave from the first sector
// boundary on (element `head`), the few before it and after the last four one by one: 58M
// elements at odd offsets 177 us, stored directly 196, aligned 174.
__device__ __forceinline__ bool off_sectors(const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 63) != 0;
}
template <typename T>
__device__ __forceinline__ int head_of(const T* p) {
    return int((64 - (reinterpret_cast<uintptr_t>(p) & 63)) & 63) / int(sizeof(T));
}
__device__ __forceinline__ void store_staged(const MultiChunk& t, const float* slot, int lane) {
    const int hp = head_of(t.p);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        const int i = hp + q * kQuarter + 4 * lane;
        const float x[4] = {slot[i], slot[i + 1], slot[i + 2], slot[i + 3]};
        if (q < kQ - 1 || i + 4 <= kWaveElems) store_f32<true>(t.p, 0, i, 4, x);
    }
    const int rp = (kWaveElems - hp) & 3;  // past the last four
    const int ip = lane < hp ? lane : kWaveElems - rp + lane - 32;
    if (lane < hp || (lane >= 32 && lane < 32 + rp)) *element<g_f32>(t.p, 0, ip) = slot[ip];
    if (!t.w_out) return;
    const int hw = head_of(t.w_out);
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        const int i = hw + q * kQuarter + 4 * lane;
        const float x[4] = {slot[i], slot[i + 1], slot[i + 2], slot[i + 3]};
        if (q < kQ - 1 || i + 4 <= kWaveElems) store_bf16<true>(t.w_out, 0, i, 4, x);
    }
    const int rw = (kWaveElems - hw) & 3;
    const int iw = lane < hw ? lane : kWaveElems - rw + lane - 32;
    if (lane < hw || (lane >= 32 && lane < 32 + rw))
        *element<g_u16>(t.w_out, 0, iw) = uint16_t(pack_bf16(slot[iw], 0.0f));
}
constexpr int kSlot = kWaveElems + 32;  // floats: a head's lanes read past the last element

// Largest old scale bytes that step8_wave takes: B1 * 2^(s - 15) and B2 * 2^(s - 31)
// have to be finite (moments below 2^16 and 2^32; others, and NaN blocks, go by quarters).
constexpr int kMostM = 142, kMostV = 158;

// 8-bit moments: what a wavefront's 1024 elements load.
struct Loaded8 {
    float p[kQ][4], g[kQ][4];
    uint32_t wm[kQ], wv[kQ];
};
template <int DT, bool ALL>
__device__ __forceinline__ void load8_wave(const MultiChunk& t, int i, int n, Loaded8& d) {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        const int live = ALL ? 4 : live_of(q * kQuarter + i, n);
        d.wm[q] = load_codes<ALL>(t.m, q, i, live);
        d.wv[q] = load_codes<ALL>(t.v, q, i, live);
        load_grad<DT, ALL>(t.g, q, i, live, d.g[q]);
        load_f32<ALL>(t.p, q, i, live, d.p[q]);
    }
    // keeps the loads here, in flight beside the scale bytes, ahead of the branch that
    // waits for those (of a whole wavefront; the up to three elements that a lane has left
    // over at a tensor's end are put together one by one, with a wait for each)
    asm volatile("" ::: "memory");
}

// 8-bit moments: a wavefront's elements from i on, those below n; lane q < 4 holds the
// scale bytes of quarter q, in and out. A code's value needs no scaling of its own: B1 * m
// is taken as (B1 * 2^(s - 15)) * float_of_bits(c << 20), the same real product, rounded
// once. What does not exist was loaded as zeros; its m and v stay 0 (no part of the
// block's largest).
//
// About 60 VALU instructions an element (stochastic; some of quarter rate), which HBM's time
// of about 100 hides: 202M parameters with bf16 gradients 523 us, 6.2 TB/s. The fp32 step's
// roots and divisions bound it by arithmetic instead (about 750); each quarter loaded on its
// own and general decoding and encoding for every block were the rest of that.
template <bool STOCH, bool ALL>
__device__ __forceinline__ void step8_wave(const MultiChunk& t, Loaded8& d, int i, int n, int lane,
                                           const MultiArgs& a, float mult, uint32_t key, int* lm,
                                           int* lv, float* slot) {
    const bool staged = ALL && (off_sectors(t.p) || (t.w_out && off_sectors(t.w_out)));
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        if (!ALL && q * kQuarter >= n) break;
        const float b1 = __builtin_ldexpf(a.k.b1, __builtin_amdgcn_readlane(*lm, q) - 15);
        const float b2 = __builtin_ldexpf(a.k.b2, __builtin_amdgcn_readlane(*lv, q) - 31);
        const int live = ALL ? 4 : live_of(q * kQuarter + i, n);
        float m[4], v[4];
        uint32_t r[4] = {};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int cm = (int(d.wm[q] << (24 - 8 * e)) >> 4) & int(0x87f00000u);
            const uint32_t cv =
                (e == 3 ? d.wv[q] >> 4 : d.wv[q] << (20 - 8 * e)) & 0x0ff00000u;
            const float x = d.g[q][e] * mult;
            m[e] = (b1 * __uint_as_float(uint32_t(cm))) + (a.k.b1c * x);
            v[e] = (b2 * __uint_as_float(cv)) + (a.k.b2c * (x * x));
            d.p[q][e] = new_p<false>(d.p[q][e], m[e], v[e], a);
            if (!ALL && e >= live) m[e] = v[e] = 0.0f;  // 0 * mult may be NaN
            if constexpr (STOCH) r[e] = mix((t.first + uint32_t(q * kQuarter + i + e)) ^ key);
        }
        const int sm = scale_of<true>(wave_max(top_bits(m)));
        const int sv = scale_of<false>(wave_max(top_bits(v)));
        uint32_t wm, wv;
        if (sm < 254 && sv < 254) {
            wm = pack_m<STOCH>(m, sm, r);
            wv = pack_v<STOCH>(v, sv, r);
        } else {
            const uint32_t rv[4] = {r[0] >> 16, r[1] >> 16, r[2] >> 16, r[3] >> 16};
            wm = encode4<true, STOCH>(m, sm, r);
            wv = encode4<false, STOCH>(v, sv, rv);
        }
        if (lane == q) {
            *lm = sm;
            *lv = sv;
        }
        if (staged) {
            reinterpret_cast<f32x4*>(slot)[q * 64 + lane] =
                f32x4{d.p[q][0], d.p[q][1], d.p[q][2], d.p[q][3]};
        } else {
            store_f32<ALL>(t.p, q, i, live, d.p[q]);
            if (t.w_out) store_bf16<ALL>(t.w_out, q, i, live, d.p[q]);
        }
        store_codes<ALL>(t.m, q, i, live, wm);
        store_codes<ALL>(t.v, q, i, live, wv);
    }
    if (staged) {
        wave_sync();
        store_staged(t, slot, lane);
        wave_sync();
    }
}

template <int DT>
__device__ __forceinline__ const void* grad_part(const void* g, int wave) {
    return static_cast<const char*>(g) + wave * kWaveElems * (DT == ZS_BF16 ? 2 : 4);
}

// The part of a chunk that one of its 4 wavefronts takes: every array from the
// wavefront's first element on, live the elements from there (none if not above 0).
// Moments of MS bytes.
template <int DT, int MS>
__device__ __forceinline__ MultiChunk wave_part(const MultiChunk& c, int wave) {
    MultiChunk t = c;
    t.g = grad_part<DT>(t.g, wave);
    const int base = wave * kWaveElems;
    t.p += base;
    t.m = static_cast<char*>(t.m) + base * MS;
    t.v = static_cast<char*>(t.v) + base * MS;
    t.m_scale += base / kQuarter;
    t.v_scale += base / kQuarter;
    if (t.w_out) t.w_out += base;
    t.first += uint32_t(base);
    t.live -= base;
    return t;
}

template <int DT, bool CACHED>
__global__ __launch_bounds__(kThreads) void multi32_kernel(
    const MultiChunk* __restrict__ chunks, int64_t n_chunks, MultiArgs a) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const float mult = a.grad_scale ? *a.grad_scale : 1.0f;
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const MultiChunk t = wave_part<DT, 4>(chunks[c], wave);
        if (t.live >= kWaveElems) step32_wave<DT, true, CACHED>(t, 4 * lane, t.live, a, mult);
        else if (t.live > 0) step32_wave<DT, false, CACHED>(t, 4 * lane, t.live, a, mult);
    }
}

template <int DT, bool STOCH, bool EXACT>
__global__ __launch_bounds__(kThreads) void multi8_kernel(
    const MultiChunk* __restrict__ chunks, int64_t n_chunks, MultiArgs a) {
    __shared__ __attribute__((aligned(16))) float slots[kWaves][kSlot];
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const float mult = a.grad_scale ? *a.grad_scale : 1.0f;
    for (int64_t c = blockIdx.x; c < n_chunks; c += gridDim.x) {
        const MultiChunk t = wave_part<DT, 1>(chunks[c], wave);
        const int n = t.live, i = 4 * lane;
        if (n <= 0) continue;
        const uint32_t key = STOCH ? tensor_key(a, t.tensor) : 0u;
        // lane q < 4 holds the scale bytes of quarter q
        g_u8* const ms = element<g_u8>(t.m_scale, 0, lane);
        g_u8* const vs = element<g_u8>(t.v_scale, 0, lane);
        const bool mine = lane < kQ && lane * kQuarter < n;
        int lm = 0, lv = 0;
        if (mine) {
            lm = *ms;
            lv = *vs;
        }
        bool done = false;
        if constexpr (!EXACT) {
            Loaded8 d;
            if (n >= kWaveElems) {
                load8_wave<DT, true>(t, i, n, d);
                done = __all(lm <= kMostM && lv <= kMostV);
                if (done)
                    step8_wave<STOCH, true>(t, d, i, n, lane, a, mult, key, &lm, &lv, slots[wave]);
            } else {
                load8_wave<DT, false>(t, i, n, d);
                done = __all(lm <= kMostM && lv <= kMostV);
                if (done)
                    step8_wave<STOCH, false>(t, d, i, n, lane, a, mult, key, &lm, &lv, nullptr);
            }
        }
        if (!done) {
#pragma unroll 1
            for (int q = 0; q < kQ && q * kQuarter < n; ++q) {
                int sm = __builtin_amdgcn_readlane(lm, q);
                int sv = __builtin_amdgcn_readlane(lv, q);
                step8_quarter<DT, STOCH, EXACT>(t, q, i, live_of(q * kQuarter + i, n), a, mult, key,
                                                &sm, &sv);
                if (lane == q) {
                    lm = sm;
                    lv = sv;
                }
            }
        }
        if (mine) {
            *ms = uint8_t(lm);
            *vs = uint8_t(lv);
        }
    }
}

// ------------------------------------------------------------- conversions

// N blocks of 256 elements per wavefront, all loads first. 202M codes to bf16, N = 4: 97 us,
// 6.3 TB/s (one block: 200, two: 103, eight: 97); to fp32, N = 2: 166, 6.1 TB/s (four: 180);
// fp32 to codes, N = 2: 158, 6.4 TB/s (four: 166, eight: 170).
template <bool SIGNED, int N>
__global__ __launch_bounds__(kThreads) void encode8_kernel(const float* __restrict__ x, int64_t S,
                                                           uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const uint32_t none[4] = {};
    for (int64_t base = (int64_t(blockIdx.x) * kWaves + wave) * (N * kQuarter); base < S;
         base += int64_t(gridDim.x) * kWaves * (N * kQuarter)) {
        const int n = int(S - base < (N * kQuarter) ? S - base : (N * kQuarter));
        float y[N][4];
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int live = live_of(q * kQuarter + 4 * lane, n);
            load_f32<false>(x + base, q, 4 * lane, live, y[q]);
        }
        int mine = 0;  // lane q: the scale byte of quarter q
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int live = live_of(q * kQuarter + 4 * lane, n);
            if constexpr (!SIGNED) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (y[q][e] < 0.0f) y[q][e] = __uint_as_float(0x7fc00000u);
            }
            const int s = scale_of<SIGNED>(wave_max(top_bits(y[q])));
            store_codes<false>(codes + base, q, 4 * lane, live,
                               encode4<SIGNED, false>(y[q], s, none));
            if (lane == q) mine = s;
        }
        if (lane * kQuarter < n && lane < N)
            *element<g_u8>(scales + base / kQuarter, 0, lane) = uint8_t(mine);
    }
}

template <bool SIGNED, int DT, int N>
__global__ __launch_bounds__(kThreads) void decode8_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           int64_t S, void* __restrict__ out) {
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    for (int64_t base = (int64_t(blockIdx.x) * kWaves + wave) * (N * kQuarter); base < S;
         base += int64_t(gridDim.x) * kWaves * (N * kQuarter)) {
        const int n = int(S - base < (N * kQuarter) ? S - base : (N * kQuarter));
        int mine = 0;
        if (lane * kQuarter < n && lane < N)
            mine = *element<const g_u8>(scales + base / kQuarter, 0, lane);
        uint32_t w[N];
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int live = live_of(q * kQuarter + 4 * lane, n);
            w[q] = load_codes<false>(codes + base, q, 4 * lane, live);
        }
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int live = live_of(q * kQuarter + 4 * lane, n);
            float x[4];
            decode4<SIGNED>(w[q], __builtin_amdgcn_readlane(mine, q), x);
            if constexpr (DT == ZS_F32)
                store_f32<false>(static_cast<float*>(out) + base, q, 4 * lane, live, x);
            else
                store_bf16<false>(static_cast<uint16_t*>(out) + base, q, 4 * lane, live, x);
        }
    }
}

// ------------------------------------------------------------- the norm

// Workgroups of the norm are 16 wavefronts, so that few of them fill the chip: each one
// counts itself in at the end, and additions to one address take about 12 ns apiece.
constexpr int kNormWaves = kNormThreads / 64;

// Sum of squares, in fp64, where the product of two fp32 numbers is exact and no square
// over- or underflows. Workgroup b takes kNormChunks chunks at a time; the one that
// arrives last adds all partial sums, in their order, and leaves the count at 0 for the
// next call. Nothing waits: which workgroup is last changes no result.
//
// A partial sum is one agent-scope atomic store, written through to memory that all XCDs
// share, and it has arrived there once the wait for it is over; the count goes up after
// that wait, so that whoever sees the whole count sees every sum.
//
// Bound by HBM: 217M fp32 gradients in 2,000 tensors 131 us, 6.6 TB/s, as bf16 75 us, 5.8, and
// 202M bf16 ones in 9 tensors 68 us, 6.0 (8 bytes a lane and load); 3.3M bf16 ones 6.0 us
// a call (a second launch for the final sum: 12.4). One count for all workgroups 137; 2048
// smaller workgroups 140 and, on the 3.3M, 13.8; a release with the count, which writes back
// and invalidates an XCD's whole L2 for every workgroup, 227 and 20.
template <int DT>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(
    const MultiChunk* __restrict__ chunks, int64_t n_chunks, double max_norm, NormWorkspace* ws,
    double* sumsq, float* norm_coef) {
    __shared__ double slot[kNormWaves];
    __shared__ bool last;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    // 4 wavefronts to a chunk
    for (int64_t c = int64_t(blockIdx.x) * kNormChunks + wave / kWaves; c < n_chunks;
         c += int64_t(gridDim.x) * kNormChunks) {
        const void* g = grad_part<DT>(chunks[c].g, wave % kWaves);
        const int n = chunks[c].live - (wave % kWaves) * kWaveElems;
        float x[kQ][4];
        if (n >= kWaveElems) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) load_grad<DT, true>(g, q, 4 * lane, 4, x[q]);
        } else {
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                load_grad<DT, false>(g, q, 4 * lane, live_of(q * kQuarter + 4 * lane, n), x[q]);
        }
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = __builtin_fma(double(x[q][e]), double(x[q][e]), s[e]);
    }
    const double mine = block_sum<kNormWaves>((s[0] + s[1]) + (s[2] + s[3]), slot);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&ws->partial[blockIdx.x], mine, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        last = arrive(ws);
    }
    __syncthreads();
    if (!last) return;
    double sum = 0.0;
    for (unsigned k = threadIdx.x; k < gridDim.x; k += kNormThreads)
        sum += __hip_atomic_load(&ws->partial[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sum = block_sum<kNormWaves>(sum, slot);
    if (threadIdx.x == 0) {
        *sumsq = sum;
        write_clip(sum, max_norm, norm_coef);
    }
}

__global__ __launch_bounds__(64) void clip_kernel(PtrPack sums, int D, double max_norm,
                                                  float* __restrict__ norm_coef) {
    if (threadIdx.x != 0) return;
    double s = 0.0;
    for (int r = 0; r < D; ++r) s += *static_cast<const double*>(sums.p[r]);
    write_clip(s, max_norm, norm_coef);
}

template <int DT, bool STOCH, bool EXACT>
void launch8(const MultiImage& im, const MultiArgs& a, hipStream_t stream) {
    const unsigned grid = unsigned(grid_blocks(im.n_chunks, 1));
    hipLaunchKernelGGL((multi8_kernel<DT, STOCH, EXACT>), dim3(grid), dim3(kThreads), 0, stream,
                       im.chunks, im.n_chunks, a);
}

template <int DT, bool CACHED>
void launch32(const MultiImage& im, const MultiArgs& a, hipStream_t stream) {
    const unsigned grid = unsigned(grid_blocks(im.n_chunks, 1));
    hipLaunchKernelGGL((multi32_kernel<DT, CACHED>), dim3(grid), dim3(kThreads), 0, stream,
                       im.chunks, im.n_chunks, a);
}

// Chunks of a step with fp32 moments that is taken to stay in the memory-side cache
// (256 MiB) between two steps: at up to 18 bytes an element of state, working copy and
// gradient, 1,800 chunks are at most 133 MB. By ordinary accesses against non-temporal ones,
// bf16 gradients, and in between a pass over M MB of other data that reads and writes it:
//   chunks        M = 0         128           192          256          512
//      200           -         6 |  7 us     6 |  7      13 |  7         -
//      800       15 | 17      15 | 21       15 | 20      32 | 21      28 | 21
//    1,800       27 | 36      33 | 39       44 | 39      60 | 39      48 | 39
//    3,200       45 | 62 and 82 | 65 with 512; 4,800: 77 | 91 and 112 | 94; 8,000: 171 | 150
// It pays while step and other data fit the cache together (the rule's assumption: small
// models, several lists a step) and costs 5 to 21 us where more lies between two steps.
// With 8-bit moments the gain is 5% or none.
constexpr int64_t kCachedChunks = 1800;

template <int DT>
void launch_dtype(const MultiImage& im, int state, const MultiArgs& a, bool stoch, bool exact,
                  hipStream_t stream) {
    if (state == ZS_STATE_F32) {
        im.n_chunks <= kCachedChunks ? launch32<DT, true>(im, a, stream)
                                     : launch32<DT, false>(im, a, stream);
    } else if (stoch) {
        exact ? launch8<DT, true, true>(im, a, stream) : launch8<DT, true, false>(im, a, stream);
    } else {
        exact ? launch8<DT, false, true>(im, a, stream) : launch8<DT, false, false>(im, a, stream);
    }
}

}  // namespace

hipError_t launch_multi(const MultiImage& im, int state, int dtype, MultiArgs a, bool stoch,
                        hipStream_t stream) {
    a.rbc2s = float(1.0 / double(a.k.bc2s));
    // when the update's approximations hold (new_p), and B1 and B2 can be scaled exactly
    const auto scales = [](float b) { return b == 0.0f || b >= 0x1p-60f; };
    const bool exact = !(a.k.eps * a.k.bc2s >= 0x1p-38f && a.k.eps <= 0x1p125f &&
                         scales(a.k.b1) && scales(a.k.b2));
    if (dtype == ZS_BF16) launch_dtype<ZS_BF16>(im, state, a, stoch, exact, stream);
    else launch_dtype<ZS_F32>(im, state, a, stoch, exact, stream);
    return hipGetLastError();
}

hipError_t launch_encode8(const float* x, int64_t S, bool is_signed, uint8_t* codes,
                          uint8_t* scales, hipStream_t stream) {
    const dim3 grid(unsigned(state8_grid(S, 2)));
    if (is_signed)
        hipLaunchKernelGGL((encode8_kernel<true, 2>), grid, dim3(kThreads), 0, stream, x, S, codes,
                           scales);
    else
        hipLaunchKernelGGL((encode8_kernel<false, 2>), grid, dim3(kThreads), 0, stream, x, S, codes,
                           scales);
    return hipGetLastError();
}

namespace {
template <bool SIGNED>
void launch_decode(const uint8_t* codes, const uint8_t* scales, int64_t S, int dtype, void* out,
                   hipStream_t stream) {
    if (dtype == ZS_F32)
        hipLaunchKernelGGL((decode8_kernel<SIGNED, ZS_F32, 2>), dim3(unsigned(state8_grid(S, 2))),
                           dim3(kThreads), 0, stream, codes, scales, S, out);
    else
        hipLaunchKernelGGL((decode8_kernel<SIGNED, ZS_BF16, 4>), dim3(unsigned(state8_grid(S, 4))),
                           dim3(kThreads), 0, stream, codes, scales, S, out);
}
}  // namespace

hipError_t launch_decode8(const uint8_t* codes, const uint8_t* scales, int64_t S, bool is_signed,
                          int dtype, void* out, hipStream_t stream) {
    is_signed ? launch_decode<true>(codes, scales, S, dtype, out, stream)
              : launch_decode<false>(codes, scales, S, dtype, out, stream);
    return hipGetLastError();
}

hipError_t launch_norm(const MultiImage& im, int dtype, double max_norm, double* sumsq,
                       float* norm_coef, NormWorkspace* ws, hipStream_t stream) {
    const dim3 grid(unsigned(norm_grid(im.n_chunks)));
    if (dtype == ZS_BF16)
        hipLaunchKernelGGL((norm_kernel<ZS_BF16>), grid, dim3(kNormThreads), 0, stream,
                           im.chunks, im.n_chunks, max_norm, ws, sumsq, norm_coef);
    else
        hipLaunchKernelGGL((norm_kernel<ZS_F32>), grid, dim3(kNormThreads), 0, stream,
                           im.chunks, im.n_chunks, max_norm, ws, sumsq, norm_coef);
    return hipGetLastError();
}

hipError_t launch_clip(const PtrPack& sums, int D, double max_norm, float* norm_coef,
                       hipStream_t stream) {
    hipLaunchKernelGGL(clip_kernel, dim3(1), dim3(64), 0, stream, sums, D, max_norm, norm_coef);
    return hipGetLastError();
}

}  // namespace zs

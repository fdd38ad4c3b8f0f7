// Products with few rows of a (serving: one new token, a handful at once) for gfx950: the
// weights b are read once, and that is the time.
//
// A workgroup takes `rows` rows of b, so many that 256 workgroups share b evenly (a CU reads
// about 20 bytes a nanosecond; 16 rows each left some CUs with three times as many as
// others). It first puts all of a into LDS as codes: it copies them, or quantises a's values
// itself (all its threads, 8 elements each, a block in the 16 lanes of a DPP row), which
// spares a launch. Its rows go 16 at a time to `splits` of its wavefronts, every
// wavefront every splits-th group of 4 blocks along K. A group's 8 KiB of b go straight to
// the registers of v_mfma_scale_f32_16x16x128_f8f6f4 as its first operand, the next two
// groups' under way meanwhile (a lane holds bytes 16 g to 16 g + 15 and 64 + 16 g to
// 64 + 16 g + 15, g = l / 16, of row l % 16: any order along K does if both operands have
// it); a is the second, its rows past M zeros. The sums of a group's wavefronts are added
// through LDS in their order. C in bf16 and fp32 (EXACT) as in the large products.

#include "zs_f8_dev.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kWaves = kF8FewWaves, kThreads = 64 * kWaves;
constexpr int kB = kF8Block;

// Elements [k, k + 8) of row m, those past the last column +0.
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

// 4 blocks of a lane's row of b, and their scale bytes.
struct Group {
    i32x4 lo[4], hi[4];
    uint32_t scales;
};

// SRC: 0, a in codes, or the type of its values.
template <int LDS, int SRC, int TA, int TB, int DT>
__global__ __launch_bounds__(kThreads) void few_kernel(F8Product p) {
    // the wavefronts' sums, twice; a's codes, rows 16 bytes further apart than they are long,
    // which puts the 16 rows that a wavefront reads at once on all banks; its scale bytes
    __shared__ __attribute__((aligned(16))) uint8_t whole[LDS];
    f32x4* const sums = reinterpret_cast<f32x4*>(whole);
    uint8_t* const lds = whole + kF8FewSums;
    const int M = int(p.a.rows), ld = p.blocks * kB + 16;
    uint8_t* const a_scales = lds + M * ld;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int part = wave % p.splits, mine = wave / p.splits, step = kWaves / p.splits;
    const int64_t n_first = int64_t(blockIdx.x) * p.tiles_n;  // rows of b a workgroup
    const int64_t n_end = min(n_first + p.tiles_n, p.b.rows);
    const int tiles = int((n_end - n_first + 15) / 16), groups = (p.blocks + 3) >> 2;
    // units of work, in a wavefront's order: its groups of its first 16 rows, of its next, ..
    struct Unit {
        int tile, at;
    };
    const auto advance = [&](Unit u) {
        u.at += p.splits;
        return u.at < groups ? u : Unit{u.tile + step, part};
    };
    const auto fetch = [&](Unit w) {
        Group x{};
        if (w.tile >= tiles || w.at >= groups) return x;
        const int64_t n = min(n_first + 16 * w.tile + r, n_end - 1);
        const g_u8* const codes = global<const g_u8>(p.b.codes + n * p.b.ld + 16 * g);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const ZS_GLOBAL i32x4* from = reinterpret_cast<const ZS_GLOBAL i32x4*>(
                codes + int64_t(min(4 * w.at + u, p.blocks - 1)) * kB);
            x.lo[u] = __builtin_nontemporal_load(from);
            x.hi[u] = __builtin_nontemporal_load(from + 4);
        }
        x.scales = *reinterpret_cast<const g_u32a*>(
            global<const g_u8>(p.b.scales + (n >> p.b.shift) * p.b.lds) + 4 * w.at);
        return x;
    };
    Unit ahead{mine, part};
    Group now = fetch(ahead);
    ahead = advance(ahead);
    Group next = fetch(ahead);
    ahead = advance(ahead);

    // 8 elements a thread, 4 such at a time so that their loads are under way together; the
    // 16 lanes of a block make the same trips
    const int units = M * p.blocks * 16;
    for (int u0 = int(threadIdx.x); u0 < units; u0 += 4 * kThreads) {
        int m[4], k[4];
        bool live[4];
        u32x2 w[4];
        Eight<SRC == 0 ? ZS_BF16 : SRC> x[4];
        uint8_t s[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int u = u0 + v * kThreads;
            live[v] = u < units;
            m[v] = u / (p.blocks * 16), k[v] = u - m[v] * (p.blocks * 16);
            if (!live[v]) continue;
            if constexpr (SRC == 0) {
                w[v] = *reinterpret_cast<const g_u32x2a*>(
                    global<const g_u8>(p.a.codes + m[v] * p.a.ld + 8 * k[v]));
                s[v] = global<const g_u8>(
                    p.a.scales)[(m[v] >> p.a.shift) * p.a.lds + k[v] / 16];
            } else {
                x[v] = eight_of<SRC>(p, m[v], 8 * k[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (!live[v]) continue;
            if constexpr (SRC != 0) {
                s[v] = uint8_t(scale_of(row_max(top_bits<SRC>(x[v])), TA));
                if constexpr (SRC == ZS_BF16)
                    w[v] = u32x2{four_codes<TA>(x[v].w[0], x[v].w[1], s[v]),
                                 four_codes<TA>(x[v].w[2], x[v].w[3], s[v])};
                else
                    w[v] = u32x2{
                        four_codes<TA>(x[v].f[0], x[v].f[1], x[v].f[2], x[v].f[3], s[v]),
                        four_codes<TA>(x[v].f[4], x[v].f[5], x[v].f[6], x[v].f[7], s[v])};
            }
            *reinterpret_cast<u32x2*>(lds + m[v] * ld + 8 * k[v]) = w[v];
            if ((k[v] & 15) == 0) a_scales[m[v] * p.blocks + k[v] / 16] = s[v];
        }
    }
    __syncthreads();

    const uint8_t* const row = lds + r * ld + 16 * g;
    for (int first = 0, round = 0; first < tiles; first += step, ++round) {
        f32x4 acc{0, 0, 0, 0};
        const int tile = first + mine;
        for (int at = part; at < groups && tile < tiles; at += p.splits) {
            const Group after = fetch(ahead);
            ahead = advance(ahead);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int block = 4 * at + u;
                if (block >= p.blocks) break;
                i32x8 a{};
                int sa = 1;
                if (r < M) {
                    const i32x4 lo = *reinterpret_cast<const i32x4*>(row + block * kB);
                    const i32x4 hi = *reinterpret_cast<const i32x4*>(row + block * kB + 64);
                    a = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    sa = a_scales[r * p.blocks + block];
                }
                const i32x8 b{now.lo[u][0], now.lo[u][1], now.lo[u][2], now.lo[u][3],
                              now.hi[u][0], now.hi[u][1], now.hi[u][2], now.hi[u][3]};
                const uint32_t sb = now.scales >> (8 * u);
                if constexpr (DT == ZS_BF16) {
                    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        b, a, acc, kFormat<TB>, kFormat<TA>, 0, int(sb), 0, sa);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            widen<TB>(b[2 * e], b[2 * e + 1], scale_value(sb)),
                            widen<TA>(a[2 * e], a[2 * e + 1], scale_value(uint32_t(sa))), acc, 0,
                            0, 0);
                }
            }
            now = next;
            next = after;
        }
        // a round's sums are read before the round after next writes there: a barrier is between
        f32x4* const here = sums + (round & 1) * kWaves * 64;
        here[wave * 64 + lane] = acc;
        __syncthreads();
        if (part != 0 || tile >= tiles) continue;
        f32x4 v = here[wave * 64 + lane];
        for (int w = 1; w < p.splits; ++w) v += here[(wave + w) * 64 + lane];
        const int64_t n = n_first + 16 * tile + 4 * g;
        if (r < M && n < n_end) put4<DT>(p, r, n, n_end, v);
    }
}

template <int SRC, int TA, int TB, int DT>
void launch_sized(const F8Product& p, hipStream_t stream) {
    const dim3 grid(unsigned((p.b.rows + p.tiles_n - 1) / p.tiles_n)), block(kThreads);
    if (f8_few_lds(p.a.rows, p.blocks) <= kF8FewLdsSmall)
        hipLaunchKernelGGL((few_kernel<int(kF8FewLdsSmall), SRC, TA, TB, DT>), grid, block, 0,
                           stream, p);
    else
        hipLaunchKernelGGL((few_kernel<int(kF8FewLds), SRC, TA, TB, DT>), grid, block, 0, stream,
                           p);
}
template <int SRC, int TA, int TB>
void launch_few(const F8Product& p, int dtype, hipStream_t stream) {
    if (dtype == ZS_BF16) launch_sized<SRC, TA, TB, ZS_BF16>(p, stream);
    else launch_sized<SRC, TA, TB, ZS_F32>(p, stream);
}

template <int SRC>
void launch_types(const F8Product& p, int type_a, int type_b, int dtype, hipStream_t stream) {
    if (type_a == ZS_E4M3) {
        if (type_b == ZS_E4M3) launch_few<SRC, ZS_E4M3, ZS_E4M3>(p, dtype, stream);
        else launch_few<SRC, ZS_E4M3, ZS_E5M2>(p, dtype, stream);
    } else {
        if (type_b == ZS_E4M3) launch_few<SRC, ZS_E5M2, ZS_E4M3>(p, dtype, stream);
        else launch_few<SRC, ZS_E5M2, ZS_E5M2>(p, dtype, stream);
    }
}

}  // namespace

hipError_t launch_few_f8(const F8Product& p, int src, int type_a, int type_b, int dtype,
                         hipStream_t stream) {
    if (src == 0) launch_types<0>(p, type_a, type_b, dtype, stream);
    else if (src == ZS_BF16) launch_types<ZS_BF16>(p, type_a, type_b, dtype, stream);
    else launch_types<ZS_F32>(p, type_a, type_b, dtype, stream);
    return hipGetLastError();
}

}  // namespace zs

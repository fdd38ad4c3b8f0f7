// Products with few rows of a (serving: one new token, a handful at once) for gfx950: the
// weights b are read once, and that is the time.
//
// All of a's codes have to fit LDS beside a group of b for each wavefront: 16 rows up to K = 4,864,
// 8 up to 9,856, 1 up to 79,232 (f8_plan); past that two launches of the larger products' way.
//
// A workgroup takes `rows` rows of b, so many that 256 workgroups, one a CU, share b evenly.
// Half of its wavefronts read and multiply: its rows go 16 at a time to `splits` of them, each
// of which takes every splits-th group of 4 blocks along K. A group's 8 KiB of codes go
// straight to the wavefront's own part of LDS, whole 512-byte pieces of rows at a time (loads
// of 64 bytes a row into registers reached 3 TB/s), and from there to
// v_mfma_scale_f32_16x16x128_f8f6f4 as its first operand. Where LDS has room for two groups
// (1 row up to K = 12,160, 2 up to 6,016, 4 up to 2,944, 16 up to 640) the next one is under way
// meanwhile; where it has one, a wavefront sends for the next when it has read the present one
// out, and its loads rest while it multiplies. The other half of the wavefronts first
// puts all of a into LDS as codes, while the first codes of b are under way: it copies them,
// or quantises a's values (8 elements a lane, a block in the 16 lanes of a DPP row), which
// spares a launch. a is the second operand, its rows past M zeros. The sums of a group's
// wavefronts are added through LDS in their order. C in bf16 and fp32 as in the large products.
//
// Measured, us (TB/s of codes), with 1.2 GB of weights in turn, so that they come from HBM / the
// same weights again, from the caches: 1 x 4096 x 4096 7.4 (2.3) / 6.4, 1 x 4096 x 11008 13.7
// (3.3) / 10.2, 1 x 11008 x 4096 12.8 (3.5) / 10.4, 16 x 11008 x 4096 20.4 (2.2) / 16.7,
// 1 x 32000 x 8192 50 (5.2) / 40; a plain read of 45 MB in turn takes 8.3. With one row what is left is
// the start, the launch and the first loads' way, some 4 us; with more, the loads' rests too.

#include "zs_f8_dev.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kWaves = kF8FewWaves, kThreads = 2 * 64 * kWaves;
constexpr int kB = kF8Block;

// All of a into LDS, by the threads of the workgroup's second half: 8 elements each, 4 such at
// a time so that their loads are under way together; the 16 lanes of a block make the same
// trips.
template <int SRC, int TA>
__device__ __forceinline__ void put_a(const F8Product& p, uint8_t* codes, uint8_t* scales, int ld) {
    constexpr int kHalf = kThreads / 2;
    const int row_units = p.blocks * 16, units = int(p.a.rows) * row_units;
    for (int u0 = int(threadIdx.x) - kHalf; u0 < units; u0 += 4 * kHalf) {
        int m[4], k[4];
        u32x2 w[4];
        Eight<SRC == 0 ? ZS_BF16 : SRC> x[4];
        uint8_t s[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int u = u0 + v * kHalf;
            m[v] = u / row_units, k[v] = u - m[v] * row_units;
            if (u >= units) continue;
            if constexpr (SRC == 0) {
                w[v] = *reinterpret_cast<const g_u32x2a*>(
                    global<const g_u8>(p.a.codes + m[v] * p.a.ld + 8 * k[v]));
                s[v] = global<const g_u8>(p.a.scales)[(m[v] >> p.a.shift) * p.a.lds + k[v] / 16];
            } else {
                x[v] = eight_of<SRC>(p, m[v], 8 * k[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (u0 + v * kHalf >= units) continue;
            if constexpr (SRC != 0) {
                s[v] = uint8_t(scale_of(row_max(top_bits<SRC>(x[v])), TA));
                w[v] = eight_codes<SRC, TA>(x[v], s[v]);
            }
            *reinterpret_cast<u32x2*>(codes + m[v] * ld + 8 * k[v]) = w[v];
            if ((k[v] & 15) == 0) scales[m[v] * p.blocks + k[v] / 16] = s[v];
        }
    }
}

// DEPTH: groups of b that a wavefront has in LDS. SRC: 0, a in codes, or the type of its
// values.
template <int DEPTH, int SRC, int TA, int TB, int DT>
__global__ __launch_bounds__(kThreads) void few_kernel(F8Product p) {
    // groups of b, each 16 rows of 512 codes and of 4 scale bytes; the wavefronts' sums, twice;
    // a's codes, rows 16 bytes further apart than they are long, which puts the 16 rows that
    // a wavefront reads at once on all banks; a's scale bytes
    __shared__ __attribute__((aligned(16))) uint8_t lds[kF8FewLds];
    constexpr int kRing = kWaves * DEPTH * int(kF8FewGroup);
    f32x4* const sums = reinterpret_cast<f32x4*>(lds + kRing);
    uint8_t* const a_codes = lds + kRing + kF8FewSums;
    const int M = int(p.a.rows), ld = p.blocks * kB + 16;
    uint8_t* const a_scales = a_codes + M * ld;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    if (wave >= kWaves) {
        put_a<SRC, TA>(p, a_codes, a_scales, ld);
        __syncthreads();
        return;
    }
    const int r = lane & 15, g = lane >> 4;
    const int part = wave % p.splits, mine = wave / p.splits, step = kWaves / p.splits;
    const int64_t n_first = int64_t(blockIdx.x) * p.tiles_n;  // tiles_n rows of b a workgroup
    const int64_t n_end = min(n_first + p.tiles_n, p.b.rows);
    const int tiles = int((n_end - n_first + 15) / 16), groups = (p.blocks + 3) >> 2;
    // units of work, in a wavefront's order: its groups of its first 16 rows, of its next, ..
    struct Unit {
        int tile, at;
    };
    const auto valid = [&](Unit u) { return u.tile < tiles && u.at < groups; };
    const auto advance = [&](Unit u) {
        u.at += p.splits;
        return u.at < groups ? u : Unit{u.tile + step, part};
    };
    // Row k of a group lies in LDS with its 16-byte pieces at j ^ k. A load takes two rows.
    uint8_t* const ring = lds + wave * DEPTH * int(kF8FewGroup);
    const uint32_t ring_at = lds_address(ring);
    const auto send = [&](Unit u, int slot) {
        const int64_t n = n_first + 16 * u.tile;
        const int last = int(n_end - n) - 1;
        const uint8_t* const base = p.b.codes + n * p.b.ld;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int row = 2 * k + (lane >> 5), piece = (lane & 31) ^ row;
            // past the last block of K its last bytes again, past the last row that row
            const int64_t col = min(int64_t(u.at) * 512 + 16 * piece, p.b.ld - 16);
            load_to_lds(base, uint32_t(min(row, last) * p.b.ld + col),
                        ring_at + slot * int(kF8FewGroup) + k * 1024);
        }
        const int in_block = int(n & ((1 << p.b.shift) - 1));
        load4_to_lds(p.b.scales + (n >> p.b.shift) * p.b.lds + 4 * u.at,
                     uint32_t(((in_block + min(r, last)) >> p.b.shift) * p.b.lds),
                     ring_at + slot * int(kF8FewGroup) + 8192);
    };
    constexpr int kLoads = 9;
    Unit ahead{mine, part};
    if (valid(ahead)) send(ahead, 0);
    if (DEPTH == 2) {
        ahead = advance(ahead);
        if (valid(ahead)) send(ahead, 1);
    }
    __syncthreads();  // all of a is there

    const uint8_t* const row = a_codes + r * ld + 32 * g;
    int slot = 0;
    for (int first = 0, round = 0; first < tiles; first += step, ++round) {
        f32x4 acc{0, 0, 0, 0};
        const int tile = first + mine;
        for (int at = part; at < groups && tile < tiles; at += p.splits) {
            if (DEPTH == 2 && valid(ahead)) arrived_but<kLoads>();
            else arrived();
            const uint8_t* const from = ring + slot * int(kF8FewGroup);
            const uint32_t scales = *reinterpret_cast<const uint32_t*>(from + 8192 + 4 * r);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int block = 4 * at + u;
                if (block >= p.blocks) break;
                i32x8 a{};
                int sa = 1;
                if (r < M) {
                    const i32x4 lo = *reinterpret_cast<const i32x4*>(row + block * kB);
                    const i32x4 hi = *reinterpret_cast<const i32x4*>(row + block * kB + 16);
                    a = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                    sa = a_scales[r * p.blocks + block];
                }
                const int piece = 8 * u + 2 * g;
                const i32x4 lo = *reinterpret_cast<const i32x4*>(from + r * 512 + (piece ^ r) * 16);
                const i32x4 hi =
                    *reinterpret_cast<const i32x4*>(from + r * 512 + ((piece + 1) ^ r) * 16);
                const i32x8 b{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                const uint32_t sb = scales >> (8 * u);
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
            ahead = advance(ahead);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot is read out
            if (valid(ahead)) send(ahead, slot);
            slot = DEPTH == 2 ? slot ^ 1 : 0;
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
    if (f8_few_lds(2, p.a.rows, p.blocks) <= kF8FewLds)
        hipLaunchKernelGGL((few_kernel<2, SRC, TA, TB, DT>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((few_kernel<1, SRC, TA, TB, DT>), grid, block, 0, stream, p);
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

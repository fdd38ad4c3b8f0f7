// Products of block-scaled 8-bit matrices, C[m, n] = sum_k a[m, k] b[n, k], for gfx950.
//
// What bounds it: the matrix cores. One product of two codes costs them half of what one in
// bf16 does, and 256 x 256 of C take 64 KiB of codes a step of 128 along K from L2 for
// 8.4 million products, so that memory stays behind.
//
// A workgroup sums a TM x TN tile of C (256, 128 or 64 squared, by 8 or 4 wavefronts) over its
// part of K. Codes go from memory straight to LDS, 16 bytes a lane, into a ring of 4 half steps
// of 64 along K: a half step multiplies what the one before read into registers, reads its
// successor's codes and sends for those of the fourth half step on, so that a load has three to
// arrive and the wait for it leaves the younger ones under way (whole steps in two buffers
// reached 2,472 TFLOP/s where this reaches 2,530; registers and LDS hold no more). The
// accumulators take 256 x 256 / 512 = 128 registers of each lane. Rows lie in LDS in pieces of
// 16 bytes, piece j of row r at j ^ (r / 4 mod 4), so that the reads of 32 rows spread over the
// banks (conflicts take 0.5 % of the CUs' cycles at 8192 x 8192 x 8192).
//
// C in bf16: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies with both scale bytes. Of 8
// neighbouring products it drops what is below 2^-13 of the largest one's power of two
// (measured; the sums of the eights are added in fp32): on normal data 2^-16 of the results'
// norm, 2^7 below the rounding to bf16, and 2^-14.5 where a few columns are much larger than
// the others, to either side alike. One result in 40 or fewer is then bf16's other neighbour
// of the exact sum; the error against 64 bits stays the rounding's (1.6572e-3 of the norm for
// 1.6568e-3). C in fp32 (EXACT): the codes, times their scales, become bf16
// exactly and v_mfma_f32_32x32x16_bf16 sums them in fp32, at half of the rate.
//
// Measured on normal data, the same operands again (C in bf16 / fp32): 8192 x 8192 x 8192 434 us,
// 2,530 TFLOP/s / 785 us, 1,400; 11008 x 4096 x 4096 169 us, 2,190 / 287 us, 1,290;
// 512 x 11008 x 4096 36 us; the same card's library in bf16 takes 664 and 393 us for the first two.
// Other cards: 478 / 833 us and, with other operands in turn, 185 / 318, the library 818 for the
// first. On zeros the first takes 340 us (3,230 TFLOP/s; 621 us in fp32): at 8192, where every
// round of tiles fills the CUs, the power that the matrix cores draw bounds it, the clock falls to
// about 1.75 GHz. 11008 x 4096 is 688 tiles on 256 CUs, three rounds for 2.69 rounds' work: a step
// of 128 costs 1.76 us there for 1.70 (on zeros 1.46 for 1.33), and the last round, with 80 CUs
// idle, up to a tenth of the time. Wavefronts of 128 x 128 (4 a workgroup) had the same rate
// and a longer epilogue.
//
// The matrix instruction's first operand is b and its second a: a lane then holds 4
// neighbouring columns n of C, which reach memory through LDS in whole lines. Tiles that leave
// CUs idle split K: each workgroup writes its partial sum, and the one that counts in last adds
// all of them in their order, so that results do not depend on who that is.

#include "zs_f8_dev.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

constexpr int kB = kF8Block;
constexpr int kMakers = 1024;  // threads of a workgroup that makes a's codes

typedef float f32x16 __attribute__((ext_vector_type(16)));

// TM x TN of C by WM x WN wavefronts, in 32 x 32 parts.
template <int TM_, int TN_, int WM_, int WN_>
struct Shape {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, W = WM * WN, kThreads = 64 * W;
    static constexpr int PM = TM / WM, PN = TN / WN, MI = PM / 32, NI = PN / 32;
    // LDS: a ring of 4 half steps (64 codes of each row of both operands), and twice the
    // scale bytes of 4 steps
    static constexpr int kHalfRow = 64, kLds = 4 * (TM + TN) * kHalfRow + 2 * (TM + TN) * 4;
    // where a's codes are made on the way: the ring is b's, all of a's codes stand behind it, by
    // half steps too, and its scale bytes, by 4 steps
    static constexpr int kMadeCodes = 4 * TN * kHalfRow + 2 * TN * 4;
    static constexpr int kMadeScales = kMadeCodes + kF8MadeBlocks * 2 * TM * kHalfRow;
    static constexpr int kMadeLds = kMadeScales + kF8MadeBlocks * TM;
    static constexpr bool kSplits = TM < 256;  // these may split K
    static_assert(TM % (16 * W) == 0 && TN % (16 * W) == 0 && TM % 64 == 0 && TN % 64 == 0 &&
                      PM % 32 == 0 && PN % 32 == 0,
                  "whole loads and parts");
};

// a's codes of a tile into LDS from its values x, by all kThreads threads of the workgroup: a
// wavefront takes 512 elements at a time of each of its rows.
template <class S, int SRC, int TA, int kThreads>
__device__ __forceinline__ void make_a(const F8Product& p, int64_t m0, uint8_t* codes,
                                       uint8_t* scales) {
    constexpr int kWaves = kThreads / 64, kRows = S::TM / kWaves;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int64_t left = p.a.rows - m0;
    const int rows = left < S::TM ? int(left) : S::TM;
    for (int k = lane; k < 16 * p.blocks; k += 64) {
        Eight<SRC> x[kRows];
#pragma unroll
        for (int v = 0; v < kRows; ++v)
            if (wave + v * kWaves < rows) x[v] = eight_of<SRC>(p, m0 + wave + v * kWaves, 8 * k);
#pragma unroll
        for (int v = 0; v < kRows; ++v) {
            const int row = wave + v * kWaves;
            if (row >= rows) break;
            const uint32_t u = row_max(top_bits<SRC>(x[v]));
            const int s = scale_of(u, TA);
            const u32x2 w = __any(is_special(u, s)) ? eight_codes<SRC, TA, true>(x[v], s)
                                                    : eight_codes<SRC, TA, false>(x[v], s);
            const int piece = ((k >> 1) & 3) ^ ((row >> 2) & 3);
            *reinterpret_cast<u32x2*>(codes + ((k >> 3) * S::TM + row) * S::kHalfRow + piece * 16 +
                                      (k & 1) * 8) = w;
            if ((k & 15) == 0) scales[((k >> 6) * S::TM + row) * 4 + ((k >> 4) & 3)] = uint8_t(s);
        }
    }
}

// Workgroup `group` of p's tiles * splits. SRC: 0, a in codes, or the type of its values, whose
// codes are made first, by kThreads threads.
template <class S, int TA, int TB, int DT, int SRC = 0, int kThreads = S::kThreads>
__device__ __forceinline__ void matmul_tile(const F8Product& p, unsigned group, uint8_t* big) {
    constexpr bool EXACT = DT == ZS_F32;
    constexpr bool MADE = SRC != 0;
    constexpr int TM = S::TM, TN = S::TN, W = S::W, MI = S::MI, NI = S::NI;
    constexpr int kRowsA = MADE ? 0 : TM, kHalfRow = S::kHalfRow, kOperand = kRowsA * kHalfRow;
    constexpr int kHalf = (kRowsA + TN) * kHalfRow, kScales = 4 * kHalf;
    constexpr int kScale = (kRowsA + TN) * 4;
    // loads of a half step, a wavefront: of a, of b; and all wavefronts' loads of scales
    constexpr int kLoadsA = kRowsA / 16 / W, kLoads = kLoadsA + TN / 16 / W;
    constexpr int kScaleLoads = (kRowsA + TN) / 64;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    // Each XCD takes a run of tiles, 8 rows of tiles deep; a tile's splits are neighbours.
    const unsigned total = unsigned(p.tiles_m) * unsigned(p.tiles_n) * unsigned(p.splits);
    const unsigned xcd = group & 7u, q = total >> 3, rest = total & 7u;
    const unsigned w = xcd * q + (xcd < rest ? xcd : rest) + (group >> 3);
    const unsigned t = w / unsigned(p.splits), split = w - t * unsigned(p.splits);
    const unsigned deep = 8, band = t / (deep * p.tiles_n);
    const unsigned rows = min(deep, unsigned(p.tiles_m) - band * deep);
    const unsigned in = t - band * deep * p.tiles_n;
    const int64_t m0 = int64_t(band * deep + in % rows) * TM, n0 = int64_t(in / rows) * TN;
    const int wm = (wave % S::WM) * S::PM, wn = (wave / S::WM) * S::PN;
    const int first = int(int64_t(p.blocks) * split / p.splits);
    const int last = int(int64_t(p.blocks) * (split + 1) / p.splits) - 1;

    if constexpr (MADE) {
        if (wave >= W) {  // these only help to make a's codes (K > 0: first <= last)
            make_a<S, SRC, TA, kThreads>(p, m0, big + S::kMadeCodes, big + S::kMadeScales);
            arrived_but<0>();
            __builtin_amdgcn_s_barrier();
            return;
        }
    }

    // What this lane loads: of each half step 16 bytes of kLoads rows, 16 * W apart, first of a,
    // then of b; and the scale bytes of a row. Rows past an operand's last are its last again:
    // what they give is not stored.
    const int64_t last_a = p.a.rows - 1 - m0, last_b = p.b.rows - 1 - n0;
    uint32_t off[kLoads];
    const int piece = ((lane & 3) ^ ((lane >> 4) & 3)) * 16;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
        const bool is_a = k < kLoadsA;
        const int64_t r = 16 * ((is_a ? k : k - kLoadsA) * W + wave) + (lane >> 2);
        off[k] = is_a ? uint32_t((r < last_a ? r : last_a) * p.a.ld) + piece
                      : uint32_t((r < last_b ? r : last_b) * p.b.ld) + piece;
    }
    const uint8_t* const codes_a = p.a.codes + m0 * p.a.ld;
    const uint8_t* const codes_b = p.b.codes + n0 * p.b.ld;
    constexpr int kMine = (kScaleLoads + W - 1) / W;
    uint32_t off_s[kMine];
    const uint8_t* base_s[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int part = wave * kMine + k;  // of 64 rows: of a, then of b
        const bool is_a = part < kRowsA / 64;
        const F8Operand& x = is_a ? p.a : p.b;
        const int64_t from = is_a ? m0 : n0, end = is_a ? last_a : last_b;
        const int64_t r = 64 * (is_a ? part : part - kRowsA / 64) + lane;
        base_s[k] = x.scales + (from >> x.shift) * x.lds;
        off_s[k] = uint32_t((((r < end ? r : end) + (from & ((1 << x.shift) - 1))) >> x.shift) * x.lds);
    }
    const uint32_t lds0 = lds_address(big);
    const auto fetch = [&](int block, int half, int slot, int k) {
        const bool is_a = k < kLoadsA;
        load_to_lds((is_a ? codes_a : codes_b) + int64_t(block) * kB + half * kHalfRow, off[k],
                    lds0 + slot * kHalf + (is_a ? 0 : kOperand) +
                        ((is_a ? k : k - kLoadsA) * W + wave) * 1024);
    };
    const auto fetch_scales = [&](int word) {
#pragma unroll
        for (int k = 0; k < kMine; ++k)
            if (wave * kMine + k < kScaleLoads)
                load4_to_lds(base_s[k] + int64_t(word) * 4, off_s[k],
                             lds0 + kScales + (word & 1) * kScale + (wave * kMine + k) * 256);
    };
    // a lane's 32 codes of a half step, of row `lane % 32` of a 32-row part
    const int row = lane & 31, g = lane >> 5;
    const uint8_t* const read_a = big + (MADE ? S::kMadeCodes : 0) + (wm + row) * kHalfRow;
    const uint8_t* const read_b = big + kOperand + (wn + row) * kHalfRow;
    const auto part = [&](const uint8_t* from, int i) {
        const uint8_t* x = from + i * 32 * kHalfRow;
        const int swap = (row >> 2) & 3;
        const i32x4 lo = *reinterpret_cast<const i32x4*>(x + (((2 * g) ^ swap) * 16));
        const i32x4 hi = *reinterpret_cast<const i32x4*>(x + (((2 * g + 1) ^ swap) * 16));
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    f32x16 acc[NI][MI] = {};
    uint32_t sa[MI], sb[NI];
    i32x8 a0[MI], b0[NI], a1[MI], b1[NI];
    // half: of all half steps, in `slot` of the ring
    const auto read = [&](int half, int slot, i32x8 (&a)[MI], i32x8 (&b)[NI]) {
        const uint8_t* const from_a = read_a + (MADE ? half * TM * kHalfRow : slot * kHalf);
        const uint8_t* const from_b = read_b + slot * kHalf;
#pragma unroll
        for (int i = 0; i < (MI > NI ? MI : NI); ++i) {
            if (i < MI) a[i] = part(from_a, i);
            if (i < NI) b[i] = part(from_b, i);
        }
    };
    const auto read_scales = [&](int k, uint32_t (&x)[MI], uint32_t (&y)[NI]) {
        const uint8_t* from = big + kScales + ((k >> 2) & 1) * kScale + row * 4;
        const uint8_t* from_a = MADE ? big + S::kMadeScales + (k >> 2) * TM * 4 + row * 4 : from;
        const int byte = 8 * (k & 3);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            x[i] = *reinterpret_cast<const uint32_t*>(from_a + (wm + 32 * i) * 4) >> byte;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            y[i] = *reinterpret_cast<const uint32_t*>(from + (kRowsA + wn + 32 * i) * 4) >> byte;
    };
    const auto multiply = [&](const i32x8 (&a)[MI], const i32x8 (&b)[NI]) {
        if constexpr (!EXACT) {
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        b[j], a[i], acc[j][i], kFormat<TB>, kFormat<TA>, 0, int(sb[j]), 0,
                        int(sa[i]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bf16x8 h[MI];
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    h[i] = widen<TA>(a[i][2 * e], a[i][2 * e + 1], scale_value(sa[i]));
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const bf16x8 y = widen<TB>(b[j][2 * e], b[j][2 * e + 1], scale_value(sb[j]));
#pragma unroll
                    for (int i = 0; i < MI; ++i)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(y, h[i], acc[j][i], 0, 0, 0);
                }
            }
        }
    };
    if (first <= last) {
        fetch_scales(first >> 2);
        fetch_scales(min((first >> 2) + 1, last >> 2));
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) fetch(min(first + (h >> 1), last), h & 1, h, k);
        if constexpr (MADE)
            make_a<S, SRC, TA, kThreads>(p, m0, big + S::kMadeCodes, big + S::kMadeScales);
        arrived_but<3 * kLoads>();
        __builtin_amdgcn_s_barrier();
        read(2 * first, 0, a0, b0);
        read_scales(first, sa, sb);
    }
    // A half step multiplies what was read in the one before, reads the next one's codes and,
    // into the slot read before, sends for those of four half steps on, so that a load has three
    // half steps to arrive. Past the last step the last one is loaded and read again: the
    // loop's body has no branches.
#pragma unroll 1
    for (int k = first; k <= last; ++k) {
        if ((k & 3) == 0) fetch_scales(min((k >> 2) + 1, last >> 2));
        const int two = 2 * ((k - first) & 1), then = min(k + 2, last);
        arrived_but<2 * kLoads>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) fetch(then, 0, two, u);
        read(2 * k + 1, two + 1, a1, b1);
        multiply(a0, b0);
        __builtin_amdgcn_sched_barrier(0);
        arrived_but<2 * kLoads>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) fetch(then, 1, two + 1, u);
        uint32_t ta[MI], tb[NI];
        read(2 * min(k + 1, last), two ^ 2, a0, b0);
        read_scales(min(k + 1, last), ta, tb);
        multiply(a1, b1);
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = ta[i];
#pragma unroll
        for (int i = 0; i < NI; ++i) sb[i] = tb[i];
        __builtin_amdgcn_sched_barrier(0);
    }
    arrived();
    __builtin_amdgcn_s_barrier();

    if (S::kSplits && !MADE && p.splits > 1) {
        // partial sums as the lanes hold them, written through to memory that all XCDs share;
        // the workgroup that counts in last adds them in their order
        typedef uint64_t u64x8 __attribute__((ext_vector_type(8)));
        const int64_t size = TM * TN / 2;  // of a partial sum, in 8 bytes
        uint64_t* const all = reinterpret_cast<uint64_t*>(p.partial) +
                              int64_t(t) * p.splits * size + wave * (MI * NI * 512) + lane;
        uint64_t* const mine = all + split * size;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const u64x8 v = __builtin_bit_cast(u64x8, acc[j][i]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    __hip_atomic_store(&mine[((j * MI + i) * 8 + e) * 64], v[e], __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        // LDS is free here: the loads of codes are over and read
        const auto flag = (ZS_LDS volatile uint32_t*)(big);
        if (threadIdx.x == 0) {
            uint32_t* const n = p.counts + t;
            const bool last_one = __hip_atomic_fetch_add(n, 1u, __ATOMIC_RELAXED,
                                                         __HIP_MEMORY_SCOPE_AGENT) + 1 ==
                                  uint32_t(p.splits);
            if (last_one) __hip_atomic_store(n, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *flag = last_one;
        }
        __syncthreads();
        if (*flag == 0) return;
        __syncthreads();  // the flag is read before its place is written again
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int i = 0; i < MI; ++i) acc[j][i] = f32x16{};
        const uint64_t* from = all;
        for (int s = 0; s < p.splits; ++s, from += size)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    u64x8 v;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = __hip_atomic_load(&from[((j * MI + i) * 8 + e) * 64],
                                                 __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    acc[j][i] += __builtin_bit_cast(f32x16, v);
                }
    }
    if (!MADE && DT == ZS_BF16 && p.accumulate) {  // the old value is added before the one rounding
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + wm + 32 * i + row;
            if (m >= p.a.rows) continue;
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t n = n0 + wn + 32 * j + 8 * e + 4 * g;
                    if (n < p.b.rows)
                        put4<DT>(p, m, n, p.b.rows,
                                 f32x4{acc[j][i][4 * e], acc[j][i][4 * e + 1],
                                       acc[j][i][4 * e + 2], acc[j][i][4 * e + 3]});
                }
        }
        return;
    }
    // Through LDS, so that C is written in whole lines: a wavefront's PM rows of up to 128 bytes
    // (64 columns in bf16, 32 in fp32) at a time, 16-byte pieces permuted by the row against
    // bank conflicts.
    constexpr int kPerPiece = DT == ZS_BF16 ? 8 : 4;
    constexpr int kCols = 8 * kPerPiece < S::PN ? 8 * kPerPiece : S::PN, kParts = kCols / 32;
    constexpr int kPieces = kCols / kPerPiece, kRows = 64 / kPieces, kRowBytes = 16 * kPieces;
    static_assert(W * S::PM * kRowBytes <= S::kLds && NI % kParts == 0, "a wavefront's rows fit");
    uint8_t* const slot = big + wave * S::PM * kRowBytes;
    const auto place = [&](int r, int at) {
        return slot + r * kRowBytes + (at ^ ((r / (16 / kPieces)) & (kPieces - 1))) * 16;
    };
#pragma unroll
    for (int j0 = 0; j0 < NI; j0 += kParts) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = 32 * i + row;
#pragma unroll
            for (int j = j0; j < j0 + kParts; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v0 = acc[j][i][4 * e], v1 = acc[j][i][4 * e + 1];
                    const float v2 = acc[j][i][4 * e + 2], v3 = acc[j][i][4 * e + 3];
                    if constexpr (DT == ZS_BF16)
                        *reinterpret_cast<u32x2*>(place(r, 4 * (j - j0) + e) + g * 8) =
                            u32x2{pack_bf16(v0, v1), pack_bf16(v2, v3)};
                    else
                        *reinterpret_cast<f32x4*>(place(r, 2 * e + g)) = f32x4{v0, v1, v2, v3};
                }
        }
#pragma unroll 4
        for (int k = 0; k < S::PM / kRows; ++k) {
            const int r = kRows * k + lane / kPieces, piece = lane % kPieces;
            const int64_t m = m0 + wm + r, n = n0 + wn + 32 * j0 + kPerPiece * piece;
            const u32x4 v = *reinterpret_cast<const u32x4*>(place(r, piece));
            if (m >= p.a.rows || n >= p.b.rows) continue;
            if constexpr (DT == ZS_BF16) {
                g_u16* c = global<g_u16>(p.c) + m * p.ldc + n;
                if (n + 8 <= p.b.rows) {
                    *reinterpret_cast<g_u32x4*>(c) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (n + e < p.b.rows) c[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
                }
            } else {
                put4<DT>(p, m, n, p.b.rows, __builtin_bit_cast(f32x4, v));
            }
        }
    }
}

template <class S, int TA, int TB, int DT>
__global__ __launch_bounds__(S::kThreads, 1) void matmul_kernel(F8Product p) {
    __shared__ __attribute__((aligned(16))) uint8_t big[S::kLds];
    matmul_tile<S, TA, TB, DT>(p, blockIdx.x, big);
}
// Two products in one launch: the first one's workgroups, then the second one's, which fill
// what those leave idle at their end.
template <class S, int TA, int TB, int DT>
__global__ __launch_bounds__(S::kThreads, 1) void matmul2_kernel(F8Product one, F8Product two,
                                                                 unsigned groups1) {
    __shared__ __attribute__((aligned(16))) uint8_t big[S::kLds];
    const bool is_one = blockIdx.x < groups1;
    matmul_tile<S, TA, TB, DT>(is_one ? one : two, is_one ? blockIdx.x : blockIdx.x - groups1, big);
}

// One whose a is given by values: a linear layer in one launch. All of a's codes stay in LDS,
// the ring is b's alone; 16 wavefronts make the codes, while the first of b are under way, and
// the 4 that multiply stay. Making them is bound by VALU instructions, some 2.7 us for K = 1024
// (f8_made has what that means against two launches).
template <class S, int SRC, int TA, int TB, int DT>
__global__ __launch_bounds__(kMakers) void linear_kernel(F8Product p) {
    __shared__ __attribute__((aligned(16))) uint8_t big[S::kMadeLds];
    matmul_tile<S, TA, TB, DT, SRC, kMakers>(p, blockIdx.x, big);
}

unsigned groups_of(const F8Product& p) {
    return unsigned(int64_t(p.tiles_m) * p.tiles_n * p.splits);
}

// two: or nullptr
template <class S, int TA, int TB>
void launch_shape(const F8Product& p, const F8Product* two, int dtype, hipStream_t stream) {
    const dim3 block(S::kThreads);
    const unsigned n = groups_of(p);
    if (two == nullptr) {
        if (dtype == ZS_BF16)
            hipLaunchKernelGGL((matmul_kernel<S, TA, TB, ZS_BF16>), dim3(n), block, 0, stream, p);
        else
            hipLaunchKernelGGL((matmul_kernel<S, TA, TB, ZS_F32>), dim3(n), block, 0, stream, p);
    } else {
        const dim3 grid(n + groups_of(*two));
        if (dtype == ZS_BF16)
            hipLaunchKernelGGL((matmul2_kernel<S, TA, TB, ZS_BF16>), grid, block, 0, stream, p,
                               *two, n);
        else
            hipLaunchKernelGGL((matmul2_kernel<S, TA, TB, ZS_F32>), grid, block, 0, stream, p, *two,
                               n);
    }
}

template <int TA, int TB>
void launch_types(const F8Product& p, const F8Product* two, int side, int dtype,
                  hipStream_t stream) {
    if (side == 256) launch_shape<Shape<256, 256, 2, 4>, TA, TB>(p, two, dtype, stream);
    else if (side == 128) launch_shape<Shape<128, 128, 2, 2>, TA, TB>(p, two, dtype, stream);
    else launch_shape<Shape<64, 64, 2, 2>, TA, TB>(p, two, dtype, stream);
}

using Made = Shape<64, 64, 2, 2>;
static_assert(kF8MadeSide == 64 && Made::kMadeLds <= 163840, "one workgroup's LDS");

template <int SRC, int TA, int TB>
void launch_linear(const F8Product& p, int dtype, hipStream_t stream) {
    const dim3 grid(groups_of(p)), block(kMakers);
    if (dtype == ZS_BF16)
        hipLaunchKernelGGL((linear_kernel<Made, SRC, TA, TB, ZS_BF16>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((linear_kernel<Made, SRC, TA, TB, ZS_F32>), grid, block, 0, stream, p);
}
template <int SRC>
void launch_linear_types(const F8Product& p, int type_a, int type_b, int dtype,
                         hipStream_t stream) {
    if (type_a == ZS_E4M3) {
        if (type_b == ZS_E4M3) launch_linear<SRC, ZS_E4M3, ZS_E4M3>(p, dtype, stream);
        else launch_linear<SRC, ZS_E4M3, ZS_E5M2>(p, dtype, stream);
    } else {
        if (type_b == ZS_E4M3) launch_linear<SRC, ZS_E5M2, ZS_E4M3>(p, dtype, stream);
        else launch_linear<SRC, ZS_E5M2, ZS_E5M2>(p, dtype, stream);
    }
}

}  // namespace

hipError_t launch_linear_f8(const F8Product& p, int src, int type_a, int type_b, int dtype,
                            hipStream_t stream) {
    if (src == ZS_BF16) launch_linear_types<ZS_BF16>(p, type_a, type_b, dtype, stream);
    else launch_linear_types<ZS_F32>(p, type_a, type_b, dtype, stream);
    return hipGetLastError();
}

hipError_t launch_matmul_f8(const F8Product& p, const F8Product* two, int side, int type_a,
                            int type_b, int dtype, hipStream_t stream) {
    if (type_a == ZS_E4M3) {
        if (type_b == ZS_E4M3) launch_types<ZS_E4M3, ZS_E4M3>(p, two, side, dtype, stream);
        else launch_types<ZS_E4M3, ZS_E5M2>(p, two, side, dtype, stream);
    } else {
        if (type_b == ZS_E4M3) launch_types<ZS_E5M2, ZS_E4M3>(p, two, side, dtype, stream);
        else launch_types<ZS_E5M2, ZS_E5M2>(p, two, side, dtype, stream);
    }
    return hipGetLastError();
}

}  // namespace zs

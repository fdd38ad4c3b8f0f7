// Device arithmetic of the kernels over many tensors: bf16 conversions and one AdamW
// element, in the operation order of the single-shard step. Files that include it are
// compiled with -ffp-contract=off (and say so here as well).
#pragma once

#include "zs_internal.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// bf16 bits -> fp32: exact, the 16 bits become the high half of the word.
__device__ __forceinline__ float bf16_lo(uint32_t word) { return __uint_as_float(word << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t word) { return __uint_as_float(word & 0xffff0000u); }

// Two values' bf16 bits in one word, rounded to nearest, ties to even, NaNs made quiet: by
// gfx950's conversion instruction, half an instruction a value.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 x{lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
}

// One AdamW element, in the fixed order, every operation rounded on its own.
__device__ __forceinline__ void adamw1(float& p, float& m, float& v, float g,
                                       const AdamConsts& k) {
    const float p1 = p * k.dec;
    const float m1 = (k.b1 * m) + (k.b1c * g);
    const float v1 = (k.b2 * v) + (k.b2c * (g * g));
    const float den = (__builtin_sqrtf(v1) / k.bc2s) + k.eps;
    p = p1 - (k.ss * (m1 / den));
    m = m1;
    v = v1;
}

}  // namespace
}  // namespace zs

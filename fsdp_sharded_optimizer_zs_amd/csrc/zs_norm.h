// Device code of a norm's end: partial sums of workgroups, joined in their order by the
// workgroup that arrives last, and the clip factor of the whole sum.
#pragma once

#include "zs_multi.h"

namespace zs {
namespace {

// Sum over a workgroup of WAVES wavefronts, in a fixed order, valid in thread 0.
template <int WAVES>
__device__ __forceinline__ double block_sum(double x, double* slot) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_down(x, d, 64);
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += slot[w];
    }
    return s;
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

// Counts this workgroup in; true for the last one of the grid. Workgroups count in
// groups (b mod kNormGroups), the last of each group for the group, so that the counts on
// one address are few; each count is put back to 0 by the last that adds to it.
__device__ __forceinline__ uint32_t count(uint32_t* n) {
    return __hip_atomic_fetch_add(n, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
}
__device__ __forceinline__ void clear(uint32_t* n) {
    __hip_atomic_store(n, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool arrive(NormWorkspace* ws) {
    const unsigned group = blockIdx.x % kNormGroups;
    const unsigned groups = gridDim.x < kNormGroups ? gridDim.x : kNormGroups;
    const unsigned members = (gridDim.x - group + kNormGroups - 1) / kNormGroups;
    if (count(&ws->arrived[group].n) != members) return false;
    clear(&ws->arrived[group].n);
    if (count(&ws->groups.n) != groups) return false;
    clear(&ws->groups.n);
    return true;
}

}  // namespace
}  // namespace zs

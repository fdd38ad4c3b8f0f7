// Internal interface between the entry points of zs_multi.cpp and the kernels of
// zs_multi.hip and zs_mx4.hip.
#pragma once

#include "zs_internal.h"
#include "zs_multi_grid.h"

namespace zs {

// Many tensors at once (zs_multi.cpp, zs_multi.hip): the device image of a table is an
// array of chunks, each with everything that the workgroup that takes it has to know, so
// that one scalar load stands before its data and every offset fits 32 bits.
struct MultiChunk {
    float* p;  // the tensor's arrays from the chunk's first element on
    void* m;
    void* v;
    uint8_t* m_scale;
    uint8_t* v_scale;
    uint16_t* w_out;
    const void* g;
    uint32_t first;  // the chunk's first element in its tensor, modulo 2^32
    int32_t tensor;  // the tensor's place in the table
    int32_t live;    // elements, 1 .. ZS_MULTI_CHUNK
    int32_t pad[3];
};
static_assert(sizeof(MultiChunk) == 80, "chunks are read by 16-byte aligned scalar loads");
struct MultiImage {
    const MultiChunk* chunks;  // device
    int64_t n_chunks;
};
struct MultiArgs {
    AdamConsts k;
    float rbc2s;              // 1 / k.bc2s
    const float* grad_scale;  // device, or nullptr
    uint32_t seed_lo, seed_hi;
};
constexpr unsigned kNormGroups = 16;
struct NormWorkspace {
    struct Count {  // on a cache line of its own; 0 between calls
        uint32_t n, pad[31];
    };
    Count groups;                // groups of workgroups that are done
    Count arrived[kNormGroups];  // workgroups of a group that are done
    double partial[kNormGrid];
};
static_assert(sizeof(NormWorkspace) <= ZS_NORM_WORKSPACE, "the caller's workspace holds it");
hipError_t launch_multi(const MultiImage& im, int state, int dtype, MultiArgs a, bool stoch,
                        hipStream_t stream);
hipError_t launch_encode8(const float* x, int64_t S, bool is_signed, uint8_t* codes,
                          uint8_t* scales, hipStream_t stream);
hipError_t launch_decode8(const uint8_t* codes, const uint8_t* scales, int64_t S, bool is_signed,
                          int dtype, void* out, hipStream_t stream);
hipError_t launch_norm(const MultiImage& im, int dtype, double max_norm, double* sumsq,
                       float* norm_coef, NormWorkspace* ws, hipStream_t stream);
hipError_t launch_clip(const PtrPack& sums, int D, double max_norm, float* norm_coef,
                       hipStream_t stream);
hipError_t launch_quantize_mx4(const void* src, int dtype, int64_t S, uint8_t* codes,
                               uint8_t* scales, hipStream_t stream);
hipError_t launch_gather_mx4(const PtrPack& codes, const PtrPack& scales, int D, int64_t S,
                             int dtype, void* flat, hipStream_t stream);

}  // namespace zs

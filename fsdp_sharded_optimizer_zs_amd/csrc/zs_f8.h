// Internal interface between the entry points of zs_f8.cpp and the kernels of
// zs_f8_quant.hip and zs_f8_gemm.hip.
#pragma once

#include "zs_f8_grid.h"
#include "zs_internal.h"

namespace zs {

// Where a quantised matrix goes (codes == nullptr: nowhere).
struct F8Out {
    uint8_t* codes;
    uint8_t* scales;
    int64_t ld, lds;
    int type;
};
// Quantisation of one matrix, as it is and transposed.
struct F8Quant {
    const void* x;
    int64_t ldx;
    int64_t rows, cols;
    int dtype;
    F8Out out, out_t;
};
// A matrix spread over D shards of S elements, from element `offset` on.
struct F8Shards {
    PtrPack shards;
    int64_t S, offset;
    double inv_s;  // 1 / S
};
hipError_t launch_quantize_f8(const F8Quant& q, int block_rows, hipStream_t stream);
// Two matrices in 1 x 128 blocks, in one launch.
hipError_t launch_quantize2_f8(const F8Quant& one, const F8Quant& two, hipStream_t stream);
hipError_t launch_gather_f8(const F8Quant& q, const F8Shards& src, int block_rows,
                            hipStream_t stream);
hipError_t launch_dequantize_f8(const uint8_t* codes, const uint8_t* scales, int block_rows,
                                int64_t rows, int64_t cols, int type, int dtype, void* out,
                                int64_t ldo, hipStream_t stream);

// An operand of a product.
struct F8Operand {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t rows;
    int64_t ld, lds;
    int shift;  // of a row to its row of scales: 0 or 7
};
struct F8Product {
    F8Operand a, b;
    void* c;
    int64_t ldc;
    int blocks;  // of 128 along K
    int accumulate;
    int tiles_m, tiles_n, splits;  // few rows: tiles_n is the plan's tn
    float* partial;    // splits > 1
    uint32_t* counts;  // likewise, 0 between calls
    const void* x;     // where a's codes are made on the way: its values, row r from
    int64_t ldx, cols; // element r * ldx on (of a, only rows is read then)
};
// side: of the tiles, the plan's tm. two: a second product of the same tiles and types in the
// same launch, or nullptr.
hipError_t launch_matmul_f8(const F8Product& p, const F8Product* two, int side, int type_a,
                            int type_b, int dtype, hipStream_t stream);
// Up to kF8Few rows of a; src: 0, a in codes, or the type of the values x.
hipError_t launch_few_f8(const F8Product& p, int src, int type_a, int type_b, int dtype,
                         hipStream_t stream);
// f8_made's products, of values x of type src.
hipError_t launch_linear_f8(const F8Product& p, int src, int type_a, int type_b, int dtype,
                            hipStream_t stream);

}  // namespace zs

// Entry points of the block-scaled 8-bit matrices, their products and the linear layer over
// them: host-side checks, then the launches. Nothing here allocates device memory or
// synchronizes.

#include <cmath>

#include "zs_f8.h"

#define ZS_EXPORT extern "C" __attribute__((visibility("default")))

using namespace zs;

namespace {

zs_status check_sizes(const char* who, const char* what, int64_t rows, int64_t cols) {
    if (rows < 0 || rows > kF8MaxRows || cols < 0 || cols > kF8MaxCols)
        return fail(ZS_EINVAL, "%s: %s is %lld x %lld, outside 2^31 - 1 x 2^22", who, what,
                    (long long)rows, (long long)cols);
    return ZS_OK;
}

zs_status check_type(const char* who, int32_t type) {
    if (type != ZS_E4M3 && type != ZS_E5M2)
        return fail(ZS_EUNSUPPORTED, "%s: unknown 8-bit type %d", who, type);
    return ZS_OK;
}

zs_status check_matrix(const char* who, const char* what, const zs_f8_matrix* x) {
    if (x == nullptr) return fail(ZS_EINVAL, "%s: %s is NULL", who, what);
    zs_status st = check_sizes(who, what, x->rows, x->cols);
    if (st != ZS_OK) return st;
    st = check_type(who, x->type);
    if (st != ZS_OK) return st;
    if (x->block_rows != 1 && x->block_rows != 128)
        return fail(ZS_EINVAL, "%s: %s: block_rows = %d is neither 1 nor 128", who, what,
                    x->block_rows);
    if (x->rows == 0 || x->cols == 0) return ZS_OK;
    if (x->codes == nullptr || x->scales == nullptr)
        return fail(ZS_EINVAL, "%s: %s: codes or scales is NULL", who, what);
    if (!aligned(x->codes, 16) || !aligned(x->scales, 4))
        return fail(ZS_EINVAL, "%s: %s: codes not 16-byte or scales not 4-byte aligned", who, what);
    return ZS_OK;
}

Range codes_of(const zs_f8_matrix& x) {
    return range_of(x.codes, f8_code_bytes(x.rows, x.cols), 1);
}
Range scales_of(const zs_f8_matrix& x) {
    return range_of(x.scales, f8_scale_bytes(x.rows, x.cols, x.block_rows), 1);
}
bool meets(const zs_f8_matrix& x, const Range& r) {
    return overlap(codes_of(x), r) || overlap(scales_of(x), r);
}

// rows x cols elements of dtype with a row stride, as a range (empty without elements).
zs_status check_dense(const char* who, const char* what, const void* p, int es, int64_t rows,
                      int64_t cols, int64_t ld, Range* out) {
    *out = Range{0, 0};
    if (rows == 0 || cols == 0) return ZS_OK;
    if (ld < cols) return fail(ZS_EINVAL, "%s: row stride of %s is below its columns", who, what);
    if (ld > INT64_MAX / 16 / es / rows)
        return fail(ZS_EINVAL, "%s: row stride of %s out of range", who, what);
    if (p == nullptr || !aligned(p, uintptr_t(es)))
        return fail(ZS_EINVAL, "%s: %s is NULL or not aligned to %d bytes", who, what, es);
    *out = range_of(p, (rows - 1) * ld + cols, es);
    return ZS_OK;
}

F8Out out_of(const zs_f8_matrix* x) {
    if (x == nullptr) return F8Out{nullptr, nullptr, 0, 0, ZS_E4M3};
    return F8Out{x->codes, x->scales, f8_ld(x->cols), f8_lds(x->cols), x->type};
}

// What a quantiser writes: shapes against each other, and overlaps. rows x cols: x's shape.
zs_status check_outputs(const char* who, const zs_f8_matrix* out, const zs_f8_matrix* out_t,
                        int64_t* rows, int64_t* cols) {
    if (out == nullptr && out_t == nullptr)
        return fail(ZS_EINVAL, "%s: out and out_t are both NULL", who);
    if (out != nullptr) {
        const zs_status st = check_matrix(who, "out", out);
        if (st != ZS_OK) return st;
    }
    if (out_t != nullptr) {
        const zs_status st = check_matrix(who, "out_t", out_t);
        if (st != ZS_OK) return st;
    }
    *rows = out != nullptr ? out->rows : out_t->cols;
    *cols = out != nullptr ? out->cols : out_t->rows;
    if (out != nullptr && out_t != nullptr) {
        if (out_t->rows != *cols || out_t->cols != *rows)
            return fail(ZS_EINVAL, "%s: out_t is not out's transpose in shape", who);
        if (out->block_rows != out_t->block_rows)
            return fail(ZS_EINVAL, "%s: out and out_t differ in block_rows", who);
    }
    if (f8_tiles(*rows, *cols) > (int64_t(1) << 31) - 1)
        return fail(ZS_EINVAL, "%s: the matrix has too many elements", who);
    const zs_f8_matrix* both[2] = {out, out_t};
    for (const zs_f8_matrix* x : both)
        if (x != nullptr && overlap(codes_of(*x), scales_of(*x)))
            return fail(ZS_EALIAS, "%s: codes and scales overlap", who);
    if (out != nullptr && out_t != nullptr &&
        (meets(*out, codes_of(*out_t)) || meets(*out, scales_of(*out_t))))
        return fail(ZS_EALIAS, "%s: out and out_t overlap", who);
    return ZS_OK;
}

int block_rows_of(const zs_f8_matrix* out, const zs_f8_matrix* out_t) {
    return (out != nullptr ? out : out_t)->block_rows;
}

// A matrix of 1 x 128 blocks in a workspace, from `at` on, which moves past it.
zs_f8_matrix place(uint8_t*& at, int64_t rows, int64_t cols, int type) {
    const auto take = [&](int64_t bytes) {
        uint8_t* p = at;
        at += f8_ceil(bytes, 256) * 256;
        return p;
    };
    zs_f8_matrix x{nullptr, nullptr, rows, cols, type, 1};
    x.codes = take(f8_code_bytes(rows, cols));
    x.scales = take(f8_scale_bytes(rows, cols, 1));
    return x;
}
int64_t placed_bytes(int64_t rows, int64_t cols) {
    return f8_ceil(f8_code_bytes(rows, cols), 256) * 256 +
           f8_ceil(f8_scale_bytes(rows, cols, 1), 256) * 256;
}

// Layout of every workspace: counts, the partial sums of the call's products, then quantised
// operands.
int64_t partial_bytes(int64_t M, int64_t N, int64_t K) {
    const int64_t n = f8_matmul_workspace(M, N, K);
    return n > 0 ? f8_ceil(n - kF8CountBytes, 256) * 256 : 0;
}

zs_status check_workspace(const char* who, const void* workspace, int64_t bytes) {
    if (bytes > 0 && (workspace == nullptr || !aligned(workspace, 16)))
        return fail(ZS_EINVAL, "%s: workspace is NULL or not 16-byte aligned", who);
    return ZS_OK;
}

F8Operand operand(const zs_f8_matrix& x) {
    return F8Operand{x.codes, x.scales, x.rows, f8_ld(x.cols), f8_lds(x.cols),
                     x.block_rows == 1 ? 0 : 7};
}

// A checked product as the kernels take it.
F8Product product_of(const zs_f8_matrix& a, const zs_f8_matrix& b, void* c, int64_t ldc,
                     int accumulate, const F8Plan& plan, uint32_t* counts, void* partial) {
    F8Product p{};
    p.a = operand(a);
    p.b = operand(b);
    p.c = c;
    p.ldc = ldc;
    p.blocks = int(f8_ceil(a.cols, kF8Block));
    p.accumulate = accumulate;
    p.tiles_m = int(plan.tiles_m);
    p.tiles_n = plan.tm == kF8Few ? plan.tn : int(plan.tiles_n);
    p.splits = plan.splits;
    p.counts = counts;
    p.partial = static_cast<float*>(partial);
    return p;
}

hipError_t product(const zs_f8_matrix& a, const zs_f8_matrix& b, int dtype, void* c, int64_t ldc,
                   int accumulate, uint32_t* counts, void* partial, hipStream_t stream) {
    const F8Plan plan = f8_plan(a.rows, b.rows, a.cols);
    const F8Product p = product_of(a, b, c, ldc, accumulate, plan, counts, partial);
    if (plan.tm == kF8Few) return launch_few_f8(p, 0, a.type, b.type, dtype, stream);
    return launch_matmul_f8(p, nullptr, plan.tm, a.type, b.type, dtype, stream);
}

// Few rows and small layers make their codes on the way and place none. (Small layers do not
// count either: theirs is the least that a layer of more than kF8Few rows asks for.)
int64_t linear_bytes(int64_t M, int64_t N, int64_t K) {
    const F8Plan plan = f8_plan(M, N, K);
    if (plan.tm == kF8Few) return 0;
    if (f8_made(plan, K)) return kF8CountBytes;
    return kF8CountBytes + partial_bytes(M, N, K) + placed_bytes(M, K);
}

int64_t groups_of(const F8Plan& p) { return p.tiles_m * p.tiles_n * p.splits; }

zs_status check_product_size(const char* who, int64_t M, int64_t N) {
    if (f8_ceil(M, 64) * f8_ceil(N, 64) > kMaxGrid)
        return fail(ZS_EINVAL, "%s: the product has too many elements", who);
    return ZS_OK;
}

}  // namespace

ZS_EXPORT zs_status zs_f8_layout(int64_t rows, int64_t cols, int32_t block_rows,
                                 int64_t* code_bytes, int64_t* scale_bytes) {
    const char* who = "zs_f8_layout";
    const zs_status st = check_sizes(who, "the matrix", rows, cols);
    if (st != ZS_OK) return st;
    if (block_rows != 1 && block_rows != 128)
        return fail(ZS_EINVAL, "%s: block_rows = %d is neither 1 nor 128", who, block_rows);
    if (!code_bytes || !scale_bytes) return fail(ZS_EINVAL, "%s: an output pointer is NULL", who);
    *code_bytes = f8_code_bytes(rows, cols);
    *scale_bytes = f8_scale_bytes(rows, cols, block_rows);
    return ok();
}

ZS_EXPORT zs_status zs_quantize_f8(const void* x, int32_t dtype, int64_t ldx,
                                   const zs_f8_matrix* out, const zs_f8_matrix* out_t,
                                   hipStream_t stream) {
    const char* who = "zs_quantize_f8";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    int64_t rows, cols;
    zs_status st = check_outputs(who, out, out_t, &rows, &cols);
    if (st != ZS_OK) return st;
    Range rx;
    st = check_dense(who, "x", x, es, rows, cols, ldx, &rx);
    if (st != ZS_OK) return st;
    if (rows == 0 || cols == 0) return ok();
    if ((out != nullptr && meets(*out, rx)) || (out_t != nullptr && meets(*out_t, rx)))
        return fail(ZS_EALIAS, "%s: x overlaps an output", who);
    const F8Quant q{x, ldx, rows, cols, dtype, out_of(out), out_of(out_t)};
    return hip_status(launch_quantize_f8(q, block_rows_of(out, out_t), stream), who);
}

ZS_EXPORT zs_status zs_gather_matrix_f8(const void* const* shards, int32_t D, int64_t S,
                                        int32_t dtype, int64_t offset, const zs_f8_matrix* out,
                                        const zs_f8_matrix* out_t, hipStream_t stream) {
    const char* who = "zs_gather_matrix_f8";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    if (D < 1 || D > ZS_MAX_D) return fail(ZS_EINVAL, "%s: D = %d outside 1..%d", who, D, ZS_MAX_D);
    if (!size_ok(S, es) || S > (int64_t(1) << 53) / D)
        return fail(ZS_EINVAL, "%s: S = %lld out of range", who, (long long)S);
    int64_t rows, cols;
    zs_status st = check_outputs(who, out, out_t, &rows, &cols);
    if (st != ZS_OK) return st;
    if (offset < 0 || offset > S * D || rows * cols > S * D - offset)
        return fail(ZS_EINVAL, "%s: elements [%lld, %lld + %lld) are not all in the unit", who,
                    (long long)offset, (long long)offset, (long long)(rows * cols));
    if (rows == 0 || cols == 0) return ok();
    F8Shards src{};
    st = take_ptrs(shards, D, es, "zs_gather_matrix_f8: shards", &src.shards);
    if (st != ZS_OK) return st;
    src.S = S;
    src.offset = offset;
    src.inv_s = 1.0 / double(S);
    for (int r = 0; r < D; ++r) {
        const Range x = range_of(src.shards.p[r], S, es);
        if ((out != nullptr && meets(*out, x)) || (out_t != nullptr && meets(*out_t, x)))
            return fail(ZS_EALIAS, "%s: shard %d overlaps an output", who, r);
    }
    const F8Quant q{nullptr, cols, rows, cols, dtype, out_of(out), out_of(out_t)};
    return hip_status(launch_gather_f8(q, src, block_rows_of(out, out_t), stream), who);
}

ZS_EXPORT zs_status zs_dequantize_f8(const zs_f8_matrix* x, int32_t dtype, void* out, int64_t ldo,
                                     hipStream_t stream) {
    const char* who = "zs_dequantize_f8";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    zs_status st = check_matrix(who, "x", x);
    if (st != ZS_OK) return st;
    if (f8_tiles(x->rows, x->cols) > (int64_t(1) << 30))
        return fail(ZS_EINVAL, "%s: the matrix has too many elements", who);
    Range ro;
    st = check_dense(who, "out", out, es, x->rows, x->cols, ldo, &ro);
    if (st != ZS_OK) return st;
    if (x->rows == 0 || x->cols == 0) return ok();
    if (meets(*x, ro)) return fail(ZS_EALIAS, "%s: out overlaps codes or scales", who);
    return hip_status(launch_dequantize_f8(x->codes, x->scales, x->block_rows, x->rows, x->cols,
                                           x->type, dtype, out, ldo, stream),
                      who);
}

ZS_EXPORT zs_status zs_matmul_f8_workspace(int64_t M, int64_t N, int64_t K, int64_t* bytes) {
    const char* who = "zs_matmul_f8_workspace";
    zs_status st = check_sizes(who, "a", M, K);
    if (st == ZS_OK) st = check_sizes(who, "b", N, K);
    if (st != ZS_OK) return st;
    if (bytes == nullptr) return fail(ZS_EINVAL, "%s: bytes is NULL", who);
    *bytes = f8_matmul_workspace(M, N, K);
    return ok();
}

ZS_EXPORT zs_status zs_matmul_f8(const zs_f8_matrix* a, const zs_f8_matrix* b, int32_t dtype,
                                 void* c, int64_t ldc, int32_t accumulate, void* workspace,
                                 hipStream_t stream) {
    const char* who = "zs_matmul_f8";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    zs_status st = check_matrix(who, "a", a);
    if (st == ZS_OK) st = check_matrix(who, "b", b);
    if (st != ZS_OK) return st;
    if (a->cols != b->cols)
        return fail(ZS_EINVAL, "%s: a has %lld columns and b %lld", who, (long long)a->cols,
                    (long long)b->cols);
    if (accumulate != 0 && accumulate != 1)
        return fail(ZS_EINVAL, "%s: accumulate must be 0 or 1", who);
    st = check_product_size(who, a->rows, b->rows);
    if (st != ZS_OK) return st;
    Range rc;
    st = check_dense(who, "c", c, es, a->rows, b->rows, ldc, &rc);
    if (st != ZS_OK) return st;
    const int64_t need = f8_matmul_workspace(a->rows, b->rows, a->cols);
    st = check_workspace(who, workspace, need);
    if (st != ZS_OK) return st;
    if (a->rows == 0 || b->rows == 0) return ok();
    const Range rw = range_of(workspace, need, 1);
    if (meets(*a, rc) || meets(*b, rc) || overlap(rc, rw))
        return fail(ZS_EALIAS, "%s: c overlaps an operand or the workspace", who);
    if (meets(*a, rw) || meets(*b, rw))
        return fail(ZS_EALIAS, "%s: the workspace overlaps an operand", who);
    return hip_status(product(*a, *b, dtype, c, ldc, accumulate, static_cast<uint32_t*>(workspace),
                              static_cast<uint8_t*>(workspace) + kF8CountBytes, stream),
                      who);
}

ZS_EXPORT zs_status zs_linear_f8_workspace(int64_t M, int64_t N, int64_t K, int64_t* bytes) {
    const char* who = "zs_linear_f8_workspace";
    zs_status st = check_sizes(who, "x", M, K);
    if (st == ZS_OK) st = check_sizes(who, "w", N, K);
    if (st != ZS_OK) return st;
    if (bytes == nullptr) return fail(ZS_EINVAL, "%s: bytes is NULL", who);
    *bytes = linear_bytes(M, N, K);
    return ok();
}

ZS_EXPORT zs_status zs_linear_f8(const void* x, int32_t dtype, int64_t M, int64_t ldx, int32_t type,
                                 const zs_f8_matrix* w, int32_t y_dtype, void* y, int64_t ldy,
                                 void* workspace, hipStream_t stream) {
    const char* who = "zs_linear_f8";
    const int es = elem_size(dtype), ys = elem_size(y_dtype);
    if (es == 0 || ys == 0)
        return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, es == 0 ? dtype : y_dtype);
    zs_status st = check_type(who, type);
    if (st == ZS_OK) st = check_matrix(who, "w", w);
    if (st != ZS_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    st = check_sizes(who, "x", M, K);
    if (st == ZS_OK) st = check_product_size(who, M, N);
    if (st == ZS_OK && f8_tiles(M, K) > (int64_t(1) << 31) - 1)
        st = fail(ZS_EINVAL, "%s: x has too many elements", who);
    Range rx, ry;
    if (st == ZS_OK) st = check_dense(who, "x", x, es, M, K, ldx, &rx);
    if (st == ZS_OK) st = check_dense(who, "y", y, ys, M, N, ldy, &ry);
    const int64_t need = linear_bytes(M, N, K);
    if (st == ZS_OK) st = check_workspace(who, workspace, need);
    if (st != ZS_OK) return st;
    if (M == 0 || N == 0) return ok();
    const Range rw = range_of(workspace, need, 1);
    if (overlap(ry, rx) || meets(*w, ry) || overlap(ry, rw))
        return fail(ZS_EALIAS, "%s: y overlaps x, w or the workspace", who);
    if (overlap(rx, rw) || meets(*w, rw))
        return fail(ZS_EALIAS, "%s: the workspace overlaps x or w", who);
    const F8Plan plan = f8_plan(M, N, K);
    if (plan.tm == kF8Few || f8_made(plan, K)) {
        const zs_f8_matrix a{nullptr, nullptr, M, K, type, 1};
        F8Product p = product_of(a, *w, y, ldy, 0, plan, nullptr, nullptr);
        p.x = x, p.ldx = ldx, p.cols = K;
        return hip_status(plan.tm == kF8Few
                              ? launch_few_f8(p, dtype, type, w->type, y_dtype, stream)
                              : launch_linear_f8(p, dtype, type, w->type, y_dtype, stream),
                          who);
    }
    uint8_t* const partial = static_cast<uint8_t*>(workspace) + kF8CountBytes;
    uint8_t* at = partial + partial_bytes(M, N, K);
    const zs_f8_matrix q = place(at, M, K, type);
    if (K > 0) {
        const hipError_t e = launch_quantize_f8(
            F8Quant{x, ldx, M, K, dtype, out_of(&q), out_of(nullptr)}, 1, stream);
        if (e != hipSuccess) return hip_status(e, who);
    }
    return hip_status(product(q, *w, y_dtype, y, ldy, 0, static_cast<uint32_t*>(workspace), partial,
                              stream),
                      who);
}

ZS_EXPORT zs_status zs_linear_f8_backward_workspace(int64_t M, int64_t N, int64_t K,
                                                    int64_t* bytes) {
    const char* who = "zs_linear_f8_backward_workspace";
    // every size is once the rows and once the columns of an operand
    const int64_t sizes[3] = {M, N, K};
    for (int64_t s : sizes) {
        const zs_status st = check_sizes(who, "an operand", s, s);
        if (st != ZS_OK) return st;
    }
    if (bytes == nullptr) return fail(ZS_EINVAL, "%s: bytes is NULL", who);
    *bytes = kF8CountBytes + partial_bytes(M, K, N) + partial_bytes(N, K, M) + placed_bytes(M, N) + placed_bytes(N, M) + placed_bytes(K, M);
    return ok();
}

ZS_EXPORT zs_status zs_linear_f8_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                          int32_t dtype, int64_t M, int64_t N, int64_t K,
                                          int32_t dy_type, const zs_f8_matrix* w_t,
                                          int32_t dx_dtype, void* dx, int64_t lddx,
                                          int32_t dw_dtype, void* dw, int64_t lddw,
                                          int32_t accumulate, void* workspace,
                                          hipStream_t stream) {
    const char* who = "zs_linear_f8_backward";
    const int es = elem_size(dtype), xs = elem_size(dx_dtype), ws = elem_size(dw_dtype);
    if (es == 0 || xs == 0 || ws == 0)
        return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d, %d or %d", who, dtype, dx_dtype,
                    dw_dtype);
    zs_status st = check_type(who, dy_type);
    if (st != ZS_OK) return st;
    if (accumulate != 0 && accumulate != 1)
        return fail(ZS_EINVAL, "%s: accumulate must be 0 or 1", who);
    int64_t need = 0;
    st = zs_linear_f8_backward_workspace(M, N, K, &need);
    if (st == ZS_OK) st = check_product_size(who, M, K);
    if (st == ZS_OK) st = check_product_size(who, N, K);
    if (st == ZS_OK && (f8_tiles(M, N) >= (int64_t(1) << 30) || f8_tiles(M, K) >= (int64_t(1) << 30)))
        st = fail(ZS_EINVAL, "%s: dy or x has too many elements", who);
    if (st != ZS_OK) return st;
    if (dx == nullptr && dw == nullptr && M > 0 && N > 0 && K > 0)
        return fail(ZS_EINVAL, "%s: dx and dw are both NULL", who);
    const bool want_dx = dx != nullptr && M > 0 && K > 0, want_dw = dw != nullptr && N > 0 && K > 0;
    Range rg, rx{0, 0}, rdx{0, 0}, rdw{0, 0};
    st = check_dense(who, "dy", dy, es, M, N, lddy, &rg);
    if (st == ZS_OK && want_dx) {
        st = check_matrix(who, "w_t", w_t);
        if (st == ZS_OK && (w_t->rows != K || w_t->cols != N))
            st = fail(ZS_EINVAL, "%s: w_t is not K x N", who);
        if (st == ZS_OK) st = check_dense(who, "dx", dx, xs, M, K, lddx, &rdx);
    }
    if (st == ZS_OK && want_dw) {
        st = check_dense(who, "x", x, es, M, K, ldx, &rx);
        if (st == ZS_OK) st = check_dense(who, "dw", dw, ws, N, K, lddw, &rdw);
    }
    if (st == ZS_OK) st = check_workspace(who, workspace, need);
    if (st != ZS_OK) return st;
    const Range rw = range_of(workspace, need, 1);
    const Range in[3] = {rg, rx, rw};
    for (const Range& r : in)
        if (overlap(rdx, r) || overlap(rdw, r))
            return fail(ZS_EALIAS, "%s: dx or dw overlaps dy, x or the workspace", who);
    if (overlap(rdx, rdw)) return fail(ZS_EALIAS, "%s: dx and dw overlap", who);
    if (overlap(rw, rg) || overlap(rw, rx))
        return fail(ZS_EALIAS, "%s: the workspace overlaps dy or x", who);
    if (want_dx && (meets(*w_t, rw) || meets(*w_t, rdx) || meets(*w_t, rdw)))
        return fail(ZS_EALIAS, "%s: w_t overlaps dx, dw or the workspace", who);

    uint8_t* const base = static_cast<uint8_t*>(workspace);
    uint32_t* const counts = static_cast<uint32_t*>(workspace);
    uint8_t* const partial = base + kF8CountBytes;
    uint8_t* const partial_dw = partial + partial_bytes(M, K, N);
    uint8_t* at = partial_dw + partial_bytes(N, K, M);
    const zs_f8_matrix g = place(at, M, N, dy_type), g_t = place(at, N, M, dy_type),
                       x_t = place(at, K, M, ZS_E4M3);
    if (M > 0 && N > 0) {
        const F8Quant from_dy{dy, lddy, M, N, dtype, out_of(want_dx ? &g : nullptr),
                              out_of(want_dw ? &g_t : nullptr)};
        const F8Quant from_x{x, ldx, M, K, dtype, out_of(nullptr), out_of(&x_t)};
        const hipError_t e = want_dw ? launch_quantize2_f8(from_dy, from_x, stream)
                                     : launch_quantize_f8(from_dy, 1, stream);
        if (e != hipSuccess) return hip_status(e, who);
    }
    // both products in one launch if they take the same kernel
    const F8Plan plan_dx = f8_plan(M, K, N), plan_dw = f8_plan(N, K, M);
    if (want_dx && want_dw && plan_dx.tm == plan_dw.tm && plan_dx.tm != kF8Few &&
        dx_dtype == dw_dtype && w_t->type == ZS_E4M3 &&
        groups_of(plan_dx) + groups_of(plan_dw) <= kMaxGrid) {
        const F8Product for_dx = product_of(g, *w_t, dx, lddx, 0, plan_dx, counts, partial);
        const F8Product for_dw = product_of(g_t, x_t, dw, lddw, accumulate, plan_dw,
                                            counts + kF8Counts, partial_dw);
        return hip_status(launch_matmul_f8(for_dx, &for_dw, plan_dx.tm, dy_type, ZS_E4M3, dx_dtype,
                                           stream),
                          who);
    }
    hipError_t e = hipSuccess;
    if (want_dx) e = product(g, *w_t, dx_dtype, dx, lddx, 0, counts, partial, stream);
    if (e == hipSuccess && want_dw)
        e = product(g_t, x_t, dw_dtype, dw, lddw, accumulate, counts + kF8Counts, partial_dw,
                    stream);
    return hip_status(e, who);
}

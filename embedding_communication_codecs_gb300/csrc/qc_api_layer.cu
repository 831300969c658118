// qc_api_layer.cu -- the C ABI of the 8-bit linear layer (declared in
// include/qcodec.h): host-side validation and dispatch.  As in qc_api.cu,
// every argument error is reported before any CUDA call.
#include <algorithm>

#include "../../include/qcodec.h"
#include "qc_api_util.h"
#include "qc_internal.h"

namespace {

using qc::api::aligned;
using qc::api::fail;
using qc::api::from_cuda;
using qc::api::ok;
using qc::api::overlaps;

size_t size_of(qc_dtype t) { return t == QC_DTYPE_F32 ? 4 : 2; }

qc_status check_dtype(const char *fn, qc_dtype t) {
    if (t != QC_DTYPE_F32 && t != QC_DTYPE_BF16)
        return fail(QC_ERR_INVALID_ARG, "%s: dtype must be QC_DTYPE_F32 or QC_DTYPE_BF16 (got %d)", fn, t);
    return QC_OK;
}

// A dimension of a layer: 1 .. QC_MAX_LAYER_DIM.
qc_status check_dim(const char *fn, const char *name, size_t v) {
    if (v < 1) return fail(QC_ERR_INVALID_ARG, "%s: %s must be positive", fn, name);
    if (v > QC_MAX_LAYER_DIM)
        return fail(QC_ERR_UNSUPPORTED, "%s: %s %zu exceeds %d", fn, name, v, QC_MAX_LAYER_DIM);
    return QC_OK;
}

// rows x dim elements, rows up to QC_MAX_LAYER_ROWS.
qc_status check_rows(const char *fn, const char *name, size_t rows, size_t dim) {
    if (rows > QC_MAX_LAYER_ROWS || rows > (static_cast<size_t>(1) << 40) / dim)
        return fail(QC_ERR_UNSUPPORTED, "%s: %s %zu x %zu exceeds %d rows or 2^40 elements", fn, name, rows,
                    dim, QC_MAX_LAYER_ROWS);
    return QC_OK;
}

// The distance between rows (rows > 0): no less than a row, and no span over 2^42 elements.
qc_status check_stride(const char *fn, const char *name, size_t stride, size_t dim, size_t rows) {
    if (stride < dim)
        return fail(QC_ERR_INVALID_ARG, "%s: %s %zu is less than the row length %zu", fn, name, stride, dim);
    if (stride > (static_cast<size_t>(1) << 42) / rows)
        return fail(QC_ERR_UNSUPPORTED, "%s: %zu rows at %s %zu span more than 2^42 elements", fn, rows, name,
                    stride);
    return QC_OK;
}

// One buffer of a call: its span in bytes, for the checks of NULL, alignment and overlap.
struct Buffer {
    const char *name;
    const void *p;
    size_t bytes;
    size_t align;
    bool output;
};

size_t span(size_t rows, size_t dim, size_t stride, size_t esize) {
    return rows == 0 ? 0 : ((rows - 1) * stride + dim) * esize;
}

// Every buffer present and aligned to its elements, no output over another buffer.
template <size_t N>
qc_status check_buffers(const char *fn, const Buffer (&b)[N]) {
    for (const Buffer &x : b) {
        if (x.bytes == 0) continue;
        if (!x.p) return fail(QC_ERR_NULL, "%s: %s is NULL", fn, x.name);
        if (!aligned(x.p, x.align))
            return fail(QC_ERR_ALIGNMENT, "%s: %s must be %zu-byte aligned", fn, x.name, x.align);
    }
    for (size_t i = 0; i < N; ++i)
        for (size_t j = i + 1; j < N; ++j)
            if ((b[i].output || b[j].output) && overlaps(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return fail(QC_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, b[i].name, b[j].name);
    return QC_OK;
}

qc_status check_workspace_size(const char *fn, size_t have, size_t need) {
    if (have < need)
        return fail(QC_ERR_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, have, need);
    return QC_OK;
}

// T, N and K of a product, and the strides of its two strided matrices.
qc_status check_product(const char *fn, size_t T, size_t N, size_t K) {
    qc_status st;
    if ((st = check_dim(fn, "N", N)) != QC_OK) return st;
    if ((st = check_dim(fn, "K", K)) != QC_OK) return st;
    if ((st = check_rows(fn, "T x N", T, N)) != QC_OK) return st;
    return check_rows(fn, "T x K", T, K);
}

cudaStream_t stream_of(qc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

#define QC_TRY(expr)                         \
    do {                                     \
        const qc_status qc_try_st = (expr);  \
        if (qc_try_st != QC_OK) return qc_try_st; \
    } while (0)

extern "C" {

qc_status qc_rowwise_int8(const void *x, qc_dtype dtype, size_t x_stride, size_t rows, size_t dim,
                          int8_t *codes, float *row_scale, qc_stream_t stream) {
    const char *fn = "qc_rowwise_int8";
    QC_TRY(check_dtype(fn, dtype));
    QC_TRY(check_dim(fn, "dim", dim));
    if (rows == 0) return ok();
    QC_TRY(check_rows(fn, "rows x dim", rows, dim));
    QC_TRY(check_stride(fn, "x_stride", x_stride, dim, rows));
    const size_t es = size_of(dtype);
    const Buffer b[] = {{"x", x, span(rows, dim, x_stride, es), es, false},
                        {"codes", codes, rows * dim, 1, true},
                        {"row_scale", row_scale, rows * 4, 4, true}};
    QC_TRY(check_buffers(fn, b));
    qc::RowCodesParams p{};
    p.x = x;
    p.x_stride = x_stride;
    p.rows = rows;
    p.dim = static_cast<uint32_t>(dim);
    p.codes = codes;
    p.row_scale = row_scale;
    return from_cuda(qc::launch_rows_int8_encode(p, dtype == QC_DTYPE_BF16, stream_of(stream)), fn);
}

qc_status qc_rowwise_int8_dequant(const int8_t *codes, const float *row_scale, size_t rows,
                                  size_t dim, void *out, qc_dtype out_dtype, size_t out_stride,
                                  qc_stream_t stream) {
    const char *fn = "qc_rowwise_int8_dequant";
    QC_TRY(check_dtype(fn, out_dtype));
    QC_TRY(check_dim(fn, "dim", dim));
    if (rows == 0) return ok();
    QC_TRY(check_rows(fn, "rows x dim", rows, dim));
    QC_TRY(check_stride(fn, "out_stride", out_stride, dim, rows));
    const size_t es = size_of(out_dtype);
    const Buffer b[] = {{"codes", codes, rows * dim, 1, false},
                        {"row_scale", row_scale, rows * 4, 4, false},
                        {"out", out, span(rows, dim, out_stride, es), es, true}};
    QC_TRY(check_buffers(fn, b));
    qc::RowCodesParams p{};
    p.codes_in = codes;
    p.scale_in = row_scale;
    p.rows = p.first_rows = rows;
    p.dim = static_cast<uint32_t>(dim);
    p.out = out;
    p.out_stride = out_stride;
    return from_cuda(qc::launch_rows_int8_decode(p, out_dtype == QC_DTYPE_BF16, stream_of(stream)), fn);
}

qc_status qc_swiglu_encode(const void *gate_up, qc_dtype dtype, size_t stride, size_t rows,
                           size_t dim, int8_t *h_codes, float *h_scale, int8_t *saved_codes,
                           float *saved_scale, qc_stream_t stream) {
    const char *fn = "qc_swiglu_encode";
    QC_TRY(check_dtype(fn, dtype));
    QC_TRY(check_dim(fn, "dim", dim));
    if (rows == 0) return ok();
    QC_TRY(check_rows(fn, "rows x (2 dim)", rows, 2 * dim));
    QC_TRY(check_stride(fn, "stride", stride, 2 * dim, rows));
    const size_t es = size_of(dtype);
    const Buffer b[] = {{"gate_up", gate_up, span(rows, 2 * dim, stride, es), es, false},
                        {"h_codes", h_codes, rows * dim, 1, true},
                        {"h_scale", h_scale, rows * 4, 4, true},
                        {"saved_codes", saved_codes, rows * 2 * dim, 1, true},
                        {"saved_scale", saved_scale, rows * 8, 4, true}};
    QC_TRY(check_buffers(fn, b));
    qc::SwigluParams p{};
    p.in = gate_up;
    p.in_stride = stride;
    p.rows = rows;
    p.dim = static_cast<uint32_t>(dim);
    p.h_codes = h_codes;
    p.h_scale = h_scale;
    p.saved_codes = saved_codes;
    p.saved_scale = saved_scale;
    p.status = qc::api::status_word();
    return from_cuda(qc::launch_swiglu_encode(p, dtype == QC_DTYPE_BF16, stream_of(stream)), fn);
}

qc_status qc_swiglu_backward(const void *dh, qc_dtype dtype, size_t dh_stride,
                             const int8_t *saved_codes, const float *saved_scale, size_t rows,
                             size_t dim, void *dgate_up, size_t dgate_up_stride,
                             qc_stream_t stream) {
    const char *fn = "qc_swiglu_backward";
    QC_TRY(check_dtype(fn, dtype));
    QC_TRY(check_dim(fn, "dim", dim));
    if (rows == 0) return ok();
    QC_TRY(check_rows(fn, "rows x (2 dim)", rows, 2 * dim));
    QC_TRY(check_stride(fn, "dh_stride", dh_stride, dim, rows));
    QC_TRY(check_stride(fn, "dgate_up_stride", dgate_up_stride, 2 * dim, rows));
    const size_t es = size_of(dtype);
    const Buffer b[] = {{"dh", dh, span(rows, dim, dh_stride, es), es, false},
                        {"saved_codes", saved_codes, rows * 2 * dim, 1, false},
                        {"saved_scale", saved_scale, rows * 8, 4, false},
                        {"dgate_up", dgate_up, span(rows, 2 * dim, dgate_up_stride, es), es, true}};
    QC_TRY(check_buffers(fn, b));
    qc::SwigluParams p{};
    p.in = dh;
    p.in_stride = dh_stride;
    p.rows = rows;
    p.dim = static_cast<uint32_t>(dim);
    p.saved_codes_in = saved_codes;
    p.saved_scale_in = saved_scale;
    p.dgate_up = dgate_up;
    p.dgate_up_stride = dgate_up_stride;
    return from_cuda(qc::launch_swiglu_backward(p, dtype == QC_DTYPE_BF16, stream_of(stream)), fn);
}

size_t qc_int8_matmul_workspace(size_t T, size_t N, size_t K) {
    if (check_product("qc_int8_matmul_workspace", T, N, K) != QC_OK) return 0;
    const size_t any = qc::int8_matmul_workspace(T, N, K, false);
    return K % 16 ? any : std::max(any, qc::int8_matmul_workspace(T, N, K, true));
}

size_t qc_int8_matmul_codes_workspace(const int8_t *x_codes, const int8_t *w_codes, size_t T, size_t N, size_t K) {
    if (check_product("qc_int8_matmul_codes_workspace", T, N, K) != QC_OK) return 0;
    return qc::int8_matmul_workspace(T, N, K, qc::wide_tokens_readable(x_codes, w_codes, K));
}

size_t qc_int8_input_grad_workspace(size_t T, size_t N, size_t K) {
    return check_product("qc_int8_input_grad_workspace", T, N, K) == QC_OK
               ? qc::int8_input_grad_workspace(T, N, K) : 0;
}

size_t qc_int8_weight_grad_workspace(size_t T, size_t N, size_t K) {
    return check_product("qc_int8_weight_grad_workspace", T, N, K) == QC_OK
               ? qc::int8_weight_grad_workspace(T, N, K) : 0;
}

qc_status qc_int8_matmul(const int8_t *x_codes, const float *x_scale, const int8_t *w_codes,
                         const float *w_scale, const float *bias, size_t T, size_t N, size_t K,
                         void *y, qc_dtype y_dtype, size_t y_stride, void *workspace,
                         size_t workspace_bytes, qc_stream_t stream) {
    const char *fn = "qc_int8_matmul";
    QC_TRY(check_dtype(fn, y_dtype));
    QC_TRY(check_product(fn, T, N, K));
    if (T == 0) return ok();
    QC_TRY(check_stride(fn, "y_stride", y_stride, N, T));
    const size_t es = size_of(y_dtype), need = qc::int8_matmul_workspace(T, N, K, qc::wide_tokens_readable(x_codes, w_codes, K));
    QC_TRY(check_workspace_size(fn, workspace_bytes, need));
    const Buffer b[] = {{"x_codes", x_codes, T * K, 1, false},
                        {"x_scale", x_scale, T * 4, 4, false},
                        {"w_codes", w_codes, N * K, 1, false},
                        {"w_scale", w_scale, N * 4, 4, false},
                        {"bias", bias, bias ? N * 4 : 0, 4, false},
                        {"y", y, span(T, N, y_stride, es), es, true},
                        {"workspace", workspace, need, 256, true}};
    QC_TRY(check_buffers(fn, b));
    qc::ProductParams p{};
    p.x_codes = x_codes;
    p.x_scale = x_scale;
    p.w_codes = w_codes;
    p.w_scale = w_scale;
    p.bias = bias;
    p.T = T;
    p.N = N;
    p.K = K;
    p.out = y;
    p.out_bf16 = y_dtype == QC_DTYPE_BF16;
    p.out_stride = y_stride;
    p.status = qc::api::status_word();
    p.workspace = workspace;
    return from_cuda(qc::launch_int8_matmul(p, stream_of(stream)), fn);
}

qc_status qc_int8_input_grad(const void *dy, size_t dy_stride, const int8_t *w_codes,
                             const float *w_scale, size_t T, size_t N, size_t K, void *dx,
                             qc_dtype dx_dtype, size_t dx_stride, void *workspace,
                             size_t workspace_bytes, qc_stream_t stream) {
    const char *fn = "qc_int8_input_grad";
    QC_TRY(check_dtype(fn, dx_dtype));
    QC_TRY(check_product(fn, T, N, K));
    if (T == 0) return ok();
    QC_TRY(check_stride(fn, "dy_stride", dy_stride, N, T));
    QC_TRY(check_stride(fn, "dx_stride", dx_stride, K, T));
    const size_t es = size_of(dx_dtype), need = qc::int8_input_grad_workspace(T, N, K);
    QC_TRY(check_workspace_size(fn, workspace_bytes, need));
    const Buffer b[] = {{"dy", dy, span(T, N, dy_stride, 2), 2, false},
                        {"w_codes", w_codes, N * K, 1, false},
                        {"w_scale", w_scale, N * 4, 4, false},
                        {"dx", dx, span(T, K, dx_stride, es), es, true},
                        {"workspace", workspace, need, 256, true}};
    QC_TRY(check_buffers(fn, b));
    qc::ProductParams p{};
    p.dy = static_cast<const uint16_t *>(dy);
    p.dy_stride = dy_stride;
    p.w_codes = w_codes;
    p.w_scale = w_scale;
    p.T = T;
    p.N = N;
    p.K = K;
    p.out = dx;
    p.out_bf16 = dx_dtype == QC_DTYPE_BF16;
    p.out_stride = dx_stride;
    p.status = qc::api::status_word();
    p.workspace = workspace;
    return from_cuda(qc::launch_int8_input_grad(p, stream_of(stream)), fn);
}

qc_status qc_int8_weight_grad(const void *dy, size_t dy_stride, const int8_t *x_codes,
                              const float *x_scale, size_t T, size_t N, size_t K, void *dw,
                              qc_dtype dw_dtype, float *dbias, int flags, void *workspace,
                              size_t workspace_bytes, qc_stream_t stream) {
    const char *fn = "qc_int8_weight_grad";
    QC_TRY(check_dtype(fn, dw_dtype));
    if (flags & ~QC_ACCUMULATE_INTO_OUT)
        return fail(QC_ERR_INVALID_ARG, "%s: flags must be 0 or QC_ACCUMULATE_INTO_OUT (got %d)", fn, flags);
    const bool accumulate = (flags & QC_ACCUMULATE_INTO_OUT) != 0;
    if (accumulate && dw_dtype != QC_DTYPE_F32)
        return fail(QC_ERR_INVALID_ARG, "%s: QC_ACCUMULATE_INTO_OUT needs an fp32 dw", fn);
    QC_TRY(check_product(fn, T, N, K));
    QC_TRY(check_rows(fn, "N x K", N, K));
    if (T > 0) QC_TRY(check_stride(fn, "dy_stride", dy_stride, N, T));
    const size_t es = size_of(dw_dtype), need = qc::int8_weight_grad_workspace(T, N, K);
    QC_TRY(check_workspace_size(fn, workspace_bytes, need));
    const Buffer b[] = {{"dy", dy, span(T, N, dy_stride, 2), 2, false},
                        {"x_codes", x_codes, T * K, 1, false},
                        {"x_scale", x_scale, T * 4, 4, false},
                        {"dw", dw, N * K * es, es, true},
                        {"dbias", dbias, dbias ? N * 4 : 0, 4, true},
                        {"workspace", workspace, need, 256, true}};
    QC_TRY(check_buffers(fn, b));
    if (T == 0 && accumulate) return ok();
    qc::ProductParams p{};
    p.dy = static_cast<const uint16_t *>(dy);
    p.dy_stride = dy_stride;
    p.x_codes = x_codes;
    p.x_scale = x_scale;
    p.T = T;
    p.N = N;
    p.K = K;
    p.out = dw;
    p.out_bf16 = dw_dtype == QC_DTYPE_BF16;
    p.out_stride = K;
    p.dbias = dbias;
    p.accumulate = accumulate;
    p.status = qc::api::status_word();
    p.workspace = workspace;
    return from_cuda(qc::launch_int8_weight_grad(p, stream_of(stream)), fn);
}

}  // extern "C"

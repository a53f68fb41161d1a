// tl_ops.cpp -- the C entry points of the operators around the product (layer
// norm, 8-bit product, orthogonalised update): argument checks, workspaces
// and launches.  The kernels are in tl_norm.cu, tl_fp8.cu and tl_ortho.cu.
#include "tiled_linear.h"
#include "tl_entry.h"
#include "tl_err_word.h"
#include "tl_fp8.h"
#include "tl_launch.h"
#include "tl_norm.h"
#include "tl_ortho.h"

#include <algorithm>
#include <climits>
#include <string>

using namespace tl;

extern "C" {

tl_status tiled_linear_operator_error_word(int32_t** word_dev) {
    return guarded([&]() -> tl_status {
        if (!word_dev) return refuse(TL_ERR_INVALID, "word_dev is null");
        *word_dev = nullptr;
        return done(operator_err_word(word_dev), "the operators' error word");
    });
}

tl_status tiled_linear_norm_forward(int64_t rows, int64_t cols, int32_t type, const void* x_dev, int64_t ldx,
                                    int32_t param_type, const void* weight_dev, const void* bias_dev, float eps,
                                    void* y_dev, int64_t ldy, float* mean_dev, float* rstd_dev,
                                    int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        NormDesc d;
        d.rows = rows;
        d.cols = cols;
        d.type = type;
        d.param_type = param_type;
        d.err = err_dev;
        d.x = x_dev;
        d.ldx = ldx;
        d.weight = weight_dev;
        d.bias = bias_dev;
        d.eps = eps;
        d.out = y_dev;
        d.ldout = ldy;
        d.mean = mean_dev;
        d.rstd = rstd_dev;
        const std::string bad = norm_check(d, false);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (rows == 0) return TL_OK;
        const int sms = device_sms();
        if (sms < 1) return refuse(TL_ERR_CUDA, "no current device");
        return done(norm_forward_launch(d, sms, static_cast<cudaStream_t>(stream)), "layer norm");
    });
}

size_t tiled_linear_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || cols > kNormMaxCols) return 0;
    return size_t(norm_partials(rows, cols)) * 2 * size_t(cols) * sizeof(float);
}

tl_status tiled_linear_norm_backward(int64_t rows, int64_t cols, int32_t type, const void* dy_dev, int64_t lddy,
                                     const void* x_dev, int64_t ldx, const float* mean_dev, const float* rstd_dev,
                                     int32_t param_type, const void* weight_dev, void* dx_dev, int64_t lddx,
                                     float* dweight_dev, float* dbias_dev, void* workspace_dev,
                                     size_t workspace_bytes, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        NormDesc d;
        d.rows = rows;
        d.cols = cols;
        d.type = type;
        d.param_type = param_type;
        d.dy = dy_dev;
        d.lddy = lddy;
        d.err = err_dev;
        d.x = x_dev;
        d.ldx = ldx;
        d.mean = const_cast<float*>(mean_dev);
        d.rstd = const_cast<float*>(rstd_dev);
        d.weight = weight_dev;
        d.out = dx_dev;
        d.ldout = lddx;
        d.dweight = dweight_dev;
        d.dbias = dbias_dev;
        d.partials = static_cast<float*>(workspace_dev);
        const std::string bad = norm_check(d, true);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (rows > 0 && (!workspace_dev || (reinterpret_cast<uintptr_t>(workspace_dev) & 15u) ||
                         workspace_bytes < tiled_linear_norm_backward_workspace_bytes(rows, cols)))
            return refuse(TL_ERR_WORKSPACE, "workspace is null, not 16-byte aligned or smaller than "
                                            "tiled_linear_norm_backward_workspace_bytes");
        const int sms = device_sms();
        if (sms < 1) return refuse(TL_ERR_CUDA, "no current device");
        return done(norm_backward_launch(d, sms, static_cast<cudaStream_t>(stream)), "layer norm backward");
    });
}

tl_status tiled_linear_fp8_quantize(int64_t rows, int64_t cols, int32_t type, const void* x_dev, int64_t ldx,
                                    int32_t format, void* row_q, int64_t ld_row, void* row_scale, void* col_q,
                                    int64_t ld_col, void* col_scale, void* tile_q, int64_t ld_tile, void* tile_scale,
                                    void* stream) {
    return guarded([&]() -> tl_status {
        Fp8QuantDesc d;
        d.rows = rows;
        d.cols = cols;
        d.type = type;
        d.x = x_dev;
        d.ldx = ldx;
        d.format = format;
        d.row = {static_cast<uint8_t*>(row_q), ld_row, static_cast<uint8_t*>(row_scale)};
        d.col = {static_cast<uint8_t*>(col_q), ld_col, static_cast<uint8_t*>(col_scale)};
        d.tile = {static_cast<uint8_t*>(tile_q), ld_tile, static_cast<uint8_t*>(tile_scale)};
        const std::string bad = fp8_quantize_check(d);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        return done(fp8_quantize_launch(d, static_cast<cudaStream_t>(stream)), "fp8 quantise");
    });
}

}  // extern "C"

namespace {

// An operand and the matrix that holds it: its own index runs down the rows or
// along the columns, and its scales are of the vectors along the reduction
// (row and col forms) or of tiles.
Fp8Operand operand(bool own_is_row, bool tiles, int64_t cols, const void* q, int64_t ld, const void* scale, int32_t format) {
    Fp8Operand o;
    o.q = q;
    o.ld = ld;
    o.mn_major = !own_is_row;
    o.format = format;
    o.scale = scale;
    o.tiles = tiles;
    o.tile_cols = (cols + kFp8Block - 1) / kFp8Block;
    return o;
}

Fp8GemmDesc product(int64_t m, int64_t n, int64_t k, const Fp8Operand& a, const Fp8Operand& b, void* d, int64_t ldd,
                    int32_t* err) {
    Fp8GemmDesc g;
    g.m_dim = m;
    g.n_dim = n;
    g.k_dim = k;
    g.a = a;
    g.b = b;
    g.d = d;
    g.ldd = ldd;
    g.err = err;
    return g;
}

tl_status launch_product(const Fp8GemmDesc& g, void* stream) {
    const int sms = device_sms();
    if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
    std::string why;
    const cudaError_t e = fp8_gemm_launch(g, sms, static_cast<cudaStream_t>(stream), &why);
    return e == cudaSuccess ? TL_OK : refuse(TL_ERR_CUDA, why);
}

tl_status fp8_product(int64_t m, int64_t n, int64_t k, const Fp8Operand& a, const Fp8Operand& b, void* d, int64_t ldd,
                      int32_t* err, void* stream) {
    const Fp8GemmDesc g = product(m, n, k, a, b, d, ldd, err);
    const std::string bad = fp8_gemm_check(g);
    return bad.empty() ? launch_product(g, stream) : refuse(TL_ERR_INVALID, bad);
}

}  // namespace

extern "C" {

tl_status tiled_linear_fp8_gemm_forward(int64_t T, int64_t K, int64_t n, int32_t x_format, const void* x_q, int64_t ldx,
                                        const void* x_scale, int32_t w_format, const void* w_q, int64_t ldw,
                                        const void* w_scale, void* y_dev, int64_t ldy, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        if (T < 0 || K < 1 || n < 1) return refuse(TL_ERR_INVALID, "T must be >= 0, K and n >= 1");
        if (T == 0) return TL_OK;
        return fp8_product(T, n, K, operand(true, false, K, x_q, ldx, x_scale, x_format),
                           operand(false, true, n, w_q, ldw, w_scale, w_format), y_dev, ldy, err_dev, stream);
    });
}

tl_status tiled_linear_fp8_gemm_dx(int64_t T, int64_t K, int64_t n, int32_t dy_format, const void* dy_q, int64_t lddy,
                                   const void* dy_scale, int32_t w_format, const void* w_q, int64_t ldw,
                                   const void* w_scale, void* dx_dev, int64_t lddx, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        if (T < 0 || K < 1 || n < 1) return refuse(TL_ERR_INVALID, "T must be >= 0, K and n >= 1");
        if (T == 0) return TL_OK;
        return fp8_product(T, K, n, operand(true, false, n, dy_q, lddy, dy_scale, dy_format),
                           operand(true, true, n, w_q, ldw, w_scale, w_format), dx_dev, lddx, err_dev, stream);
    });
}

tl_status tiled_linear_fp8_gemm_dw(int64_t T, int64_t K, int64_t n, int32_t x_format, const void* x_q, int64_t ldx,
                                   const void* x_scale, int32_t dy_format, const void* dy_q, int64_t lddy,
                                   const void* dy_scale, void* dw_dev, int64_t lddw, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        if (T < 0 || K < 1 || n < 1) return refuse(TL_ERR_INVALID, "T must be >= 0, K and n >= 1");
        if (T == 0) {
            if (!dw_dev || lddw < n) return refuse(TL_ERR_INVALID, "dw is null or its leading dimension smaller than n");
            return done(cudaMemset2DAsync(dw_dev, size_t(lddw) * 2, 0, size_t(n) * 2, size_t(K),
                                          static_cast<cudaStream_t>(stream)), "fp8 dw");
        }
        return fp8_product(K, n, T, operand(false, false, K, x_q, ldx, x_scale, x_format),
                           operand(false, false, n, dy_q, lddy, dy_scale, dy_format), dw_dev, lddw, err_dev,
                           stream);
    });
}

}  // extern "C"

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// One 8-bit form of a [rows, cols] matrix in a workspace.
struct Held {
    Fp8QuantDesc::Form form;
    size_t q_bytes = 0, scale_bytes = 0;
    Held(int64_t rows, int64_t cols, bool by_row) {
        form.ldq = (cols + 15) / 16 * 16;
        q_bytes = up256(size_t(rows) * size_t(form.ldq));
        const int64_t along = by_row ? cols : rows, vectors = by_row ? rows : cols;
        scale_bytes = up256(size_t((along + 4 * kFp8Block - 1) / (4 * kFp8Block)) * size_t(vectors) * 4);
    }
    size_t bytes() const { return q_bytes + scale_bytes; }
    uint8_t* place(uint8_t* at) {
        form.q = at;
        form.scale = at + q_bytes;
        return at + bytes();
    }
};

bool layer_ok(int64_t T, int64_t K, int64_t n) {
    return T >= 0 && K >= 1 && n >= 1 && T <= INT32_MAX / 2 && K <= INT32_MAX / 2 && n <= INT32_MAX / 2;
}

Fp8QuantDesc quantizing(int64_t rows, int64_t cols, int32_t type, const void* x, int64_t ldx, const Fp8QuantDesc::Form* row,
                        const Fp8QuantDesc::Form* col) {
    Fp8QuantDesc d;
    d.rows = rows;
    d.cols = cols;
    d.type = type;
    d.x = x;
    d.ldx = ldx;
    d.format = TL_FP8_E4M3;
    if (row) d.row = *row;
    if (col) d.col = *col;
    return d;
}
tl_status quantize(const Fp8QuantDesc& d, void* stream) {  // checked
    return done(fp8_quantize_launch(d, static_cast<cudaStream_t>(stream)), "fp8 quantise");
}

}  // namespace

extern "C" {

size_t tiled_linear_fp8_linear_workspace_bytes(int64_t T, int64_t K, int64_t n) {
    return layer_ok(T, K, n) ? Held(std::max<int64_t>(T, 1), K, true).bytes() : 0;
}

tl_status tiled_linear_fp8_linear(int64_t T, int64_t K, int64_t n, int32_t type, const void* x_dev, int64_t ldx,
                                  int32_t w_format, const void* w_q, int64_t ldw, const void* w_scale, void* y_dev,
                                  int64_t ldy, void* workspace_dev, size_t workspace_bytes, int32_t* err_dev,
                                  void* stream) {
    return guarded([&]() -> tl_status {
        if (!layer_ok(T, K, n)) return refuse(TL_ERR_INVALID, "T must be >= 0, K and n >= 1, all below 2^30");
        if (T == 0) return TL_OK;
        if (!workspace_ok(workspace_dev, workspace_bytes, tiled_linear_fp8_linear_workspace_bytes(T, K, n)))
            return refuse(TL_ERR_WORKSPACE, "workspace is null, not 256-byte aligned or too small");
        Held x(T, K, true);
        x.place(static_cast<uint8_t*>(workspace_dev));
        Fp8GemmDesc g = product(T, n, K, operand(true, false, K, x.form.q, x.form.ldq, x.form.scale, TL_FP8_E4M3),
                                operand(false, true, n, w_q, ldw, w_scale, w_format), y_dev, ldy, err_dev);
        g.early = true;  // the quantiser, directly ahead, writes x's form alone
        const Fp8QuantDesc qx = quantizing(T, K, type, x_dev, ldx, &x.form, nullptr);
        std::string bad = fp8_gemm_check(g);
        if (bad.empty()) bad = fp8_quantize_check(qx);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        const tl_status st = quantize(qx, stream);
        return st == TL_OK ? launch_product(g, stream) : st;
    });
}

size_t tiled_linear_fp8_linear_backward_workspace_bytes(int64_t T, int64_t K, int64_t n) {
    if (!layer_ok(T, K, n)) return 0;
    const int64_t t = std::max<int64_t>(T, 1);
    return Held(t, n, true).bytes() + Held(t, n, false).bytes() + Held(t, K, false).bytes();
}

tl_status tiled_linear_fp8_linear_backward(int64_t T, int64_t K, int64_t n, int32_t type, const void* x_dev,
                                           int64_t ldx, const void* dy_dev, int64_t lddy, int32_t w_format,
                                           const void* w_q, int64_t ldw, const void* w_scale, void* dx_dev,
                                           int64_t lddx, void* dw_dev, int64_t lddw, void* workspace_dev,
                                           size_t workspace_bytes, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        if (!layer_ok(T, K, n)) return refuse(TL_ERR_INVALID, "T must be >= 0, K and n >= 1, all below 2^30");
        if (!dx_dev && !dw_dev) return refuse(TL_ERR_INVALID, "neither dx nor dw is wanted");
        if (T == 0)
            return dw_dev ? tiled_linear_fp8_gemm_dw(T, K, n, 0, nullptr, 0, nullptr, 0, nullptr, 0, nullptr, dw_dev, lddw,
                                                     err_dev, stream)
                          : TL_OK;
        if (!workspace_ok(workspace_dev, workspace_bytes, tiled_linear_fp8_linear_backward_workspace_bytes(T, K, n)))
            return refuse(TL_ERR_WORKSPACE, "workspace is null, not 256-byte aligned or too small");
        Held dy_row(T, n, true), dy_col(T, n, false), x_col(T, K, false);
        x_col.place(dy_col.place(dy_row.place(static_cast<uint8_t*>(workspace_dev))));
        const auto form = [](const Held& h, bool own_is_row, int64_t cols) {
            return operand(own_is_row, false, cols, h.form.q, h.form.ldq, h.form.scale, TL_FP8_E4M3);
        };
        // everything is checked before anything is enqueued
        const Fp8GemmDesc gx = product(T, K, n, form(dy_row, true, n), operand(true, true, n, w_q, ldw, w_scale, w_format),
                                       dx_dev, lddx, err_dev);
        const Fp8GemmDesc gw = product(K, n, T, form(x_col, false, K), form(dy_col, false, n), dw_dev, lddw, err_dev);
        std::string bad = dx_dev ? fp8_gemm_check(gx) : std::string();
        if (bad.empty() && dw_dev) bad = fp8_gemm_check(gw);
        if (bad.empty() && dw_dev && (!x_dev || ldx < K)) bad = "x is null or its leading dimension is smaller than K";
        const Fp8QuantDesc qdy = quantizing(T, n, type, dy_dev, lddy, dx_dev ? &dy_row.form : nullptr, dw_dev ? &dy_col.form : nullptr);
        const Fp8QuantDesc qx = quantizing(T, K, type, x_dev, ldx, nullptr, &x_col.form);
        if (bad.empty()) bad = fp8_quantize_check(qdy);
        if (bad.empty() && dw_dev) bad = fp8_quantize_check(qx);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        tl_status st = quantize(qdy, stream);
        if (st == TL_OK && dx_dev) st = launch_product(gx, stream);
        if (st == TL_OK && dw_dev) st = quantize(qx, stream);
        if (st == TL_OK && dw_dev) st = launch_product(gw, stream);
        return st;
    });
}

size_t tiled_linear_orthogonalize_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
    return ortho_workspace(batch, rows, cols);
}

tl_status tiled_linear_orthogonalize(int64_t batch, int64_t rows, int64_t cols, int32_t type, const void* g_dev,
                                     int64_t ldg, int64_t g_apart, int32_t steps, float a, float b, float c, float eps,
                                     float scale, void* out_dev, int64_t ldo, int64_t o_apart, void* workspace_dev,
                                     size_t workspace_bytes, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        OrthoDesc d;
        d.batch = batch;
        d.rows = rows;
        d.cols = cols;
        d.type = type;
        d.g = g_dev;
        d.ldg = ldg;
        d.g_apart = g_apart;
        d.steps = steps;
        d.a = a;
        d.b = b;
        d.c = c;
        d.eps = eps;
        d.scale = scale;
        d.out = out_dev;
        d.ldo = ldo;
        d.o_apart = o_apart;
        d.workspace = workspace_dev;
        d.err = err_dev;
        const std::string bad = ortho_check(d);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (batch == 0) return TL_OK;
        if (!workspace_ok(workspace_dev, workspace_bytes, ortho_workspace(batch, rows, cols)))
            return refuse(TL_ERR_WORKSPACE, "workspace is null, not 256-byte aligned or too small");
        const int sms = device_sms();
        if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
        std::string why;
        const cudaError_t e = ortho_launch(d, sms, static_cast<cudaStream_t>(stream), &why);
        if (e == cudaSuccess) return TL_OK;
        return refuse(TL_ERR_CUDA, why.empty() ? std::string("orthogonalize: ") + cudaGetErrorString(e) : why);
    });
}

}  // extern "C"

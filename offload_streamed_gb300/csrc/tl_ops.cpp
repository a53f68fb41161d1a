// tl_ops.cpp -- the C entry points of the operators around the product (layer
// norm, 8-bit product, orthogonalised update): argument checks, workspaces
// and launches.  The kernels are in tl_norm.cu, tl_fp8.cu and tl_ortho.cu.
#include "tiled_linear.h"
#include "tl_launch.h"
#include "tl_norm.h"
#include "tl_unbound_error.h"

#include <exception>

using namespace tl;

namespace {

tl_status refuse(tl_status st, const std::string& why) {
    tl::set_unbound_error(why);
    return st;
}

tl_status done(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return TL_OK;
    return refuse(TL_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Nothing is thrown across the ABI.
template <typename F>
tl_status guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception& e) {
        return refuse(TL_ERR_STATE, e.what());
    } catch (...) {
        return refuse(TL_ERR_STATE, "unknown exception");
    }
}

}  // namespace

extern "C" {

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

}  // extern "C"

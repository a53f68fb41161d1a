// tl_row_ops.cpp -- the C entry points of the operators whose weight depends on the
// row (router, products grouped by expert, adapters): argument checks, workspaces
// and launches.  The kernels are in tl_route.cu, tl_grouped.cu, tl_grouped_dw.cu
// and tl_adapter.cu.
#include "tiled_linear.h"
#include "tl_adapter.h"
#include "tl_entry.h"
#include "tl_grouped.h"
#include "tl_launch.h"
#include "tl_route.h"

#include <algorithm>
#include <climits>
#include <string>

using namespace tl;

namespace {

const char* const kWorkspace = "workspace is null, not 256-byte aligned or too small";

RouteDesc grouping(int64_t T, int64_t k, int64_t groups, const int32_t* ids, int32_t* slots, int32_t* rows, int32_t* offsets, void* workspace) {
    RouteDesc d;
    d.tokens = T;
    d.k = k;
    d.groups = groups;
    d.ids = const_cast<int32_t*>(ids);
    d.slots = slots;
    d.rows = rows;
    d.offsets = offsets;
    d.counts = static_cast<int32_t*>(workspace);
    return d;
}

tl_status launched(cudaError_t e, const std::string& why, const char* what) {
    if (e == cudaSuccess) return TL_OK;
    return refuse(TL_ERR_CUDA, why.empty() ? std::string(what) + ": " + cudaGetErrorString(e) : why);
}

}  // namespace

extern "C" {

size_t tiled_linear_route_workspace_bytes(int64_t T, int64_t k, int64_t groups) { return route_workspace(T, k, groups); }

tl_status tiled_linear_group_rows(int64_t T, int64_t k, int64_t groups, const int32_t* ids_dev, int32_t* slots_dev, int32_t* rows_dev,
                                  int32_t* offsets_dev, void* workspace_dev, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> tl_status {
        const RouteDesc d = grouping(T, k, groups, ids_dev, slots_dev, rows_dev, offsets_dev, workspace_dev);
        const std::string bad = route_check(d, false);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (!workspace_ok(workspace_dev, workspace_bytes, route_workspace(T, k, groups))) return refuse(TL_ERR_WORKSPACE, kWorkspace);
        return done(group_rows_launch(d, static_cast<cudaStream_t>(stream)), "group rows");
    });
}

tl_status tiled_linear_route(int64_t T, int64_t experts, int64_t k, int32_t type, const void* logits_dev, int64_t ld, int32_t normalize,
                             float* weights_dev, int32_t* ids_dev, int32_t* slots_dev, int32_t* rows_dev, int32_t* offsets_dev,
                             void* workspace_dev, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> tl_status {
        RouteDesc d = grouping(T, k, experts, ids_dev, slots_dev, rows_dev, offsets_dev, workspace_dev);
        d.type = type;
        d.logits = logits_dev;
        d.ld = ld;
        d.normalize = normalize != 0;
        d.weights = weights_dev;
        const std::string bad = route_check(d, true);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (!workspace_ok(workspace_dev, workspace_bytes, route_workspace(T, k, experts))) return refuse(TL_ERR_WORKSPACE, kWorkspace);
        return done(route_launch(d, static_cast<cudaStream_t>(stream)), "route");
    });
}

tl_status tiled_linear_route_backward(int64_t T, int64_t experts, int64_t k, int32_t type, const void* logits_dev, int64_t ld,
                                      const int32_t* ids_dev, const float* dweights_dev, int32_t normalize, void* dlogits_dev, int64_t lddl,
                                      void* stream) {
    return guarded([&]() -> tl_status {
        RouteBackwardDesc d;
        d.tokens = T;
        d.k = k;
        d.experts = experts;
        d.type = type;
        d.logits = logits_dev;
        d.ld = ld;
        d.ids = ids_dev;
        d.dweights = dweights_dev;
        d.normalize = normalize != 0;
        d.dlogits = dlogits_dev;
        d.ldd = lddl;
        const std::string bad = route_backward_check(d);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        return done(route_backward_launch(d, static_cast<cudaStream_t>(stream)), "route backward");
    });
}

tl_status tiled_linear_combine(int64_t T, int64_t k, int64_t cols, int64_t rows, int32_t type, const void* y_dev, int64_t ldy,
                               const int32_t* slots_dev, const float* weights_dev, void* out_dev, int64_t ldout, void* stream) {
    return guarded([&]() -> tl_status {
        CombineDesc d;
        d.tokens = T;
        d.k = k;
        d.cols = cols;
        d.rows = rows;
        d.type = type;
        d.y = y_dev;
        d.ldy = ldy;
        d.slots = slots_dev;
        d.weights = weights_dev;
        d.out = out_dev;
        d.ldout = ldout;
        const std::string bad = combine_check(d, false);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        return done(combine_launch(d, static_cast<cudaStream_t>(stream)), "combine");
    });
}

tl_status tiled_linear_combine_backward(int64_t T, int64_t k, int64_t cols, int64_t rows, int32_t type, const void* dout_dev, int64_t lddout,
                                        const int32_t* slots_dev, const void* y_dev, int64_t ldy, const float* weights_dev, void* dy_dev,
                                        int64_t lddy, float* dweights_dev, void* stream) {
    return guarded([&]() -> tl_status {
        CombineDesc d;
        d.tokens = T;
        d.k = k;
        d.cols = cols;
        d.rows = rows;
        d.type = type;
        d.y = y_dev;
        d.ldy = ldy;
        d.slots = slots_dev;
        d.weights = weights_dev;
        d.out = dy_dev;
        d.ldout = lddy;
        d.dout = dout_dev;
        d.lddout = lddout;
        d.dweights = dweights_dev;
        const std::string bad = combine_check(d, true);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        return done(combine_backward_launch(d, static_cast<cudaStream_t>(stream)), "combine backward");
    });
}

size_t tiled_linear_grouped_workspace_bytes(int64_t R, int64_t K) {
    if (R < 0 || K < 1 || R > INT32_MAX / 2 || K > INT32_MAX / 2) return 0;
    return std::max<size_t>(256, size_t(R) * size_t(picked_ld(K)) * 2);
}

tl_status tiled_linear_grouped_forward(int64_t R, int64_t K, int64_t n, int64_t groups, int32_t type, const void* x_dev, int64_t ldx,
                                       int64_t x_rows, const int32_t* rows_dev, const void* w_dev, int64_t ldw, int64_t w_apart,
                                       const int32_t* offsets_dev, void* y_dev, int64_t ldy, void* workspace_dev, size_t workspace_bytes,
                                       int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        GroupedDesc d;
        d.rows = R;
        d.reduce = K;
        d.own = n;
        d.groups = groups;
        d.type = type;
        d.offsets = offsets_dev;
        d.x = {x_dev, ldx, x_rows, rows_dev};
        d.w = w_dev;
        d.ldw = ldw;
        d.w_apart = w_apart;
        d.own_contiguous = true;
        d.out = {y_dev, ldy, R, nullptr};
        d.err = err_dev;
        const std::string bad = grouped_check(d);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (R == 0) return TL_OK;
        if (rows_dev && !workspace_ok(workspace_dev, workspace_bytes, tiled_linear_grouped_workspace_bytes(R, K))) return refuse(TL_ERR_WORKSPACE, kWorkspace);
        d.gathered = workspace_dev;
        const int sms = device_sms();
        if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
        std::string why;
        return launched(grouped_launch(d, sms, static_cast<cudaStream_t>(stream), &why), why, "grouped product");
    });
}

tl_status tiled_linear_grouped_dx(int64_t R, int64_t K, int64_t n, int64_t groups, int32_t type, const void* dy_dev, int64_t lddy,
                                  const void* w_dev, int64_t ldw, int64_t w_apart, const int32_t* offsets_dev, void* dx_dev, int64_t lddx,
                                  int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        GroupedDesc d;
        d.rows = R;
        d.reduce = n;
        d.own = K;
        d.groups = groups;
        d.type = type;
        d.offsets = offsets_dev;
        d.x = {dy_dev, lddy, R, nullptr};
        d.w = w_dev;
        d.ldw = ldw;
        d.w_apart = w_apart;
        d.own_contiguous = false;
        d.out = {dx_dev, lddx, R, nullptr};
        d.err = err_dev;
        const std::string bad = grouped_check(d);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (R == 0) return TL_OK;
        const int sms = device_sms();
        if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
        std::string why;
        return launched(grouped_launch(d, sms, static_cast<cudaStream_t>(stream), &why), why, "grouped dx");
    });
}

tl_status tiled_linear_grouped_dw(int64_t R, int64_t K, int64_t n, int64_t groups, int32_t type, const void* x_dev, int64_t ldx, int64_t x_rows,
                                  const int32_t* rows_dev, const void* dy_dev, int64_t lddy, const int32_t* offsets_dev, void* dw_dev,
                                  int64_t lddw, int64_t dw_apart, void* workspace_dev, size_t workspace_bytes, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        GroupedDwDesc d;
        d.rows = R;
        d.m_dim = K;
        d.n_dim = n;
        d.groups = groups;
        d.type = type;
        d.offsets = offsets_dev;
        d.x = {x_dev, ldx, x_rows, rows_dev};
        d.dy = {dy_dev, lddy, R, nullptr};
        d.dw = dw_dev;
        d.lddw = lddw;
        d.dw_apart = dw_apart;
        d.err = err_dev;
        const std::string bad = grouped_dw_check(d);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (R > 0 && rows_dev && !workspace_ok(workspace_dev, workspace_bytes, tiled_linear_grouped_workspace_bytes(R, K)))
            return refuse(TL_ERR_WORKSPACE, kWorkspace);
        d.gathered = workspace_dev;
        const int sms = device_sms();
        if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
        std::string why;
        return launched(grouped_dw_launch(d, sms, static_cast<cudaStream_t>(stream), &why), why, "grouped dw");
    });
}

size_t tiled_linear_adapter_workspace_bytes(int64_t T, int64_t r, int64_t adapters) { return adapter_workspace(T, r, adapters); }

tl_status tiled_linear_adapter_forward(int64_t T, int64_t K, int64_t n, int64_t r, int64_t adapters, int32_t type, const void* x_dev, int64_t ldx,
                                       const void* a_dev, int64_t lda, int64_t a_apart, const void* b_dev, int64_t ldb, int64_t b_apart,
                                       const int32_t* ids_dev, const float* scale_dev, float scale, int32_t base_type, const void* base_dev,
                                       int64_t ldbase, void* y_dev, int64_t ldy, void* h_dev, int64_t ldh, void* workspace_dev,
                                       size_t workspace_bytes, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        AdapterDesc d;
        d.tokens = T;
        d.K = K;
        d.n = n;
        d.rank = r;
        d.adapters = adapters;
        d.type = type;
        d.x = x_dev;
        d.ldx = ldx;
        d.a = a_dev;
        d.lda = lda;
        d.a_apart = a_apart;
        d.b = b_dev;
        d.ldb = ldb;
        d.b_apart = b_apart;
        d.ids = ids_dev;
        d.scale = scale_dev;
        d.scale_all = scale;
        d.base = base_dev;
        d.base_type = base_type;
        d.ldbase = ldbase;
        d.y = y_dev;
        d.ldy = ldy;
        d.h = h_dev;
        d.ldh = ldh;
        d.workspace = workspace_dev;
        d.err = err_dev;
        const std::string bad = adapter_check(d, false);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (T == 0) return TL_OK;
        if (!workspace_ok(workspace_dev, workspace_bytes, adapter_workspace(T, r, adapters))) return refuse(TL_ERR_WORKSPACE, kWorkspace);
        const int sms = device_sms();
        if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
        std::string why;
        return launched(adapter_forward_launch(d, sms, static_cast<cudaStream_t>(stream), &why), why, "adapters");
    });
}

tl_status tiled_linear_adapter_backward(int64_t T, int64_t K, int64_t n, int64_t r, int64_t adapters, int32_t type, const void* x_dev, int64_t ldx,
                                        const void* h_dev, int64_t ldh, const void* dy_dev, int64_t lddy, const void* a_dev, int64_t lda,
                                        int64_t a_apart, const void* b_dev, int64_t ldb, int64_t b_apart, const int32_t* ids_dev,
                                        const float* scale_dev, float scale, int32_t base_type, const void* base_dev, int64_t ldbase, void* dx_dev,
                                        int64_t lddx, void* da_dev, int64_t ldda, int64_t da_apart, void* db_dev, int64_t lddb, int64_t db_apart,
                                        void* workspace_dev, size_t workspace_bytes, int32_t* err_dev, void* stream) {
    return guarded([&]() -> tl_status {
        AdapterDesc d;
        d.tokens = T;
        d.K = K;
        d.n = n;
        d.rank = r;
        d.adapters = adapters;
        d.type = type;
        d.x = x_dev;
        d.ldx = ldx;
        d.h = const_cast<void*>(h_dev);
        d.ldh = ldh;
        d.dy = dy_dev;
        d.lddy = lddy;
        d.a = a_dev;
        d.lda = lda;
        d.a_apart = a_apart;
        d.b = b_dev;
        d.ldb = ldb;
        d.b_apart = b_apart;
        d.ids = ids_dev;
        d.scale = scale_dev;
        d.scale_all = scale;
        d.base = base_dev;
        d.base_type = base_type;
        d.ldbase = ldbase;
        d.dx = dx_dev;
        d.lddx = lddx;
        d.da = da_dev;
        d.ldda = ldda;
        d.da_apart = da_apart;
        d.db = db_dev;
        d.lddb = lddb;
        d.db_apart = db_apart;
        d.workspace = workspace_dev;
        d.err = err_dev;
        const std::string bad = adapter_check(d, true);
        if (!bad.empty()) return refuse(TL_ERR_INVALID, bad);
        if (!workspace_ok(workspace_dev, workspace_bytes, adapter_workspace(T, r, adapters))) return refuse(TL_ERR_WORKSPACE, kWorkspace);
        const int sms = device_sms();
        if (sms < 2) return refuse(TL_ERR_CUDA, "no current device");
        std::string why;
        return launched(adapter_backward_launch(d, sms, static_cast<cudaStream_t>(stream), &why), why, "adapters' backward");
    });
}

}  // extern "C"

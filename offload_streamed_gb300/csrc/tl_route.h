// tl_route.h -- internal interface of the router (host side): which experts a
// token goes to, the order of its entries by expert, and the sum of the
// experts' answers.
#pragma once
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

namespace tl {

constexpr int64_t kMaxGroups = 1024;  // experts or groups
constexpr int64_t kMaxTop = 32;       // entries of a token

// Group ids [T, k] by value; with logits, find the ids first.
struct RouteDesc {
    int64_t tokens = 0, k = 0, groups = 0;
    int32_t* ids = nullptr;  // read by group_rows, written by route
    int32_t* slots = nullptr;
    int32_t* rows = nullptr;
    int32_t* offsets = nullptr;
    int32_t* counts = nullptr;  // workspace
    // route only
    int32_t type = 0;  // tl_type of the logits
    const void* logits = nullptr;
    int64_t ld = 0;
    bool normalize = true;
    float* weights = nullptr;
};
std::string route_check(const RouteDesc& d, bool with_logits);
size_t route_workspace(int64_t tokens, int64_t k, int64_t groups);
cudaError_t group_rows_launch(const RouteDesc& d, cudaStream_t stream);
cudaError_t route_launch(const RouteDesc& d, cudaStream_t stream);

struct RouteBackwardDesc {
    int64_t tokens = 0, k = 0, experts = 0;
    int32_t type = 0;  // of the logits and their gradient
    const void* logits = nullptr;
    int64_t ld = 0;
    const int32_t* ids = nullptr;
    const float* dweights = nullptr;
    bool normalize = true;
    void* dlogits = nullptr;
    int64_t ldd = 0;
};
std::string route_backward_check(const RouteBackwardDesc& d);
cudaError_t route_backward_launch(const RouteBackwardDesc& d, cudaStream_t stream);

// out[t] = sum_j weights[t, j] y[slots[t, j]] and its backward.
struct CombineDesc {
    int64_t tokens = 0, k = 0, cols = 0, rows = 0;  // rows: of y
    int32_t type = 0;
    const void* y = nullptr;
    int64_t ldy = 0;
    const int32_t* slots = nullptr;
    const float* weights = nullptr;  // nullptr: ones
    void* out = nullptr;             // [tokens, cols], or dy [rows, cols]
    int64_t ldout = 0;
    // backward only
    const void* dout = nullptr;
    int64_t lddout = 0;
    float* dweights = nullptr;  // nullptr: not wanted
};
std::string combine_check(const CombineDesc& d, bool backward);
cudaError_t combine_launch(const CombineDesc& d, cudaStream_t stream);
cudaError_t combine_backward_launch(const CombineDesc& d, cudaStream_t stream);

}  // namespace tl

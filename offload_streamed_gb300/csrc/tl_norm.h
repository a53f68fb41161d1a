// tl_norm.h -- internal interface of the layer norm (host side).
#pragma once
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

namespace tl {

// Rows longer than this are refused: eight CTAs of a cluster hold one row.
constexpr int64_t kNormMaxCols = 131072;

struct NormDesc {
    int64_t rows = 0, cols = 0;
    int32_t type = 0;        // tl_type of x, y, dy and dx
    int32_t param_type = 0;  // tl_type of weight and bias
    const void* x = nullptr;
    int64_t ldx = 0;
    const void* weight = nullptr;  // nullptr: ones
    const void* bias = nullptr;    // nullptr: zeros (forward)
    float eps = 0;
    void* out = nullptr;  // y (forward) or dx (backward)
    int64_t ldout = 0;
    float* mean = nullptr;
    float* rstd = nullptr;
    int32_t* err = nullptr;  // device word that a bounded wait sets
    // backward only
    const void* dy = nullptr;
    int64_t lddy = 0;
    float* dweight = nullptr;  // nullptr: not wanted
    float* dbias = nullptr;
    float* partials = nullptr;  // norm_partials() rows of 2 * cols floats
};

std::string norm_check(const NormDesc& d, bool backward);
cudaError_t norm_forward_launch(const NormDesc& d, int num_sms, cudaStream_t stream);
cudaError_t norm_backward_launch(const NormDesc& d, int num_sms, cudaStream_t stream);
// Most partial sums of the weight's gradient that a backward pass writes.
int64_t norm_partials(int64_t rows, int64_t cols);

}  // namespace tl

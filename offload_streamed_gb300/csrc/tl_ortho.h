// tl_ortho.h -- internal interface of the orthogonalised update (host side).
#pragma once
#include <cstddef>
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

namespace tl {

struct OrthoDesc {
    int64_t batch = 0, rows = 0, cols = 0;
    int32_t type = 0;  // tl_type of g
    const void* g = nullptr;
    int64_t ldg = 0, g_apart = 0;  // elements between rows, between matrices
    int32_t steps = 0;
    float a = 0, b = 0, c = 0, eps = 0, scale = 1;
    void* out = nullptr;  // bf16
    int64_t ldo = 0, o_apart = 0;
    void* workspace = nullptr;  // ortho_workspace() bytes, 256-byte aligned
    int32_t* err = nullptr;
};

std::string ortho_check(const OrthoDesc& d);
size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols);  // 0: invalid sizes
cudaError_t ortho_launch(const OrthoDesc& d, int num_sms, cudaStream_t stream, std::string* why);

}  // namespace tl

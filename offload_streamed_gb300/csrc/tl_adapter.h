// tl_adapter.h -- internal interface of the low-rank adapters (host side).
#pragma once
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

namespace tl {

constexpr int64_t kAdapterMaxRank = 128;

// Row t belongs to adapter ids[t] (none where that is not 0 .. adapters - 1):
//   h[t] = x[t] . a[id],   y[t] = base[t] + scale[id] h[t] . b[id]
struct AdapterDesc {
    int64_t tokens = 0, K = 0, n = 0, rank = 0, adapters = 0;
    int32_t type = 0;  // TL_TYPE_BF16 or TL_TYPE_F16
    const void* x = nullptr;
    int64_t ldx = 0;
    const void* a = nullptr;  // [adapters][K, rank]
    int64_t lda = 0, a_apart = 0;
    const void* b = nullptr;  // [adapters][rank, n]
    int64_t ldb = 0, b_apart = 0;
    const int32_t* ids = nullptr;
    const float* scale = nullptr;  // [adapters]; nullptr: scale_all
    float scale_all = 1.0f;
    const void* base = nullptr;  // as y (forward), as dx (backward); nullptr: zeros
    int32_t base_type = 0;
    int64_t ldbase = 0;
    void* h = nullptr;  // written by the forward, read by the backward
    int64_t ldh = 0;
    void* y = nullptr;
    int64_t ldy = 0;
    // backward
    const void* dy = nullptr;
    int64_t lddy = 0;
    void* dx = nullptr;  // nullptr: not wanted
    int64_t lddx = 0;
    void* da = nullptr;  // as a; nullptr: neither da nor db is wanted
    int64_t ldda = 0, da_apart = 0;
    void* db = nullptr;
    int64_t lddb = 0, db_apart = 0;
    void* workspace = nullptr;
    int32_t* err = nullptr;
};
std::string adapter_check(const AdapterDesc& d, bool backward);
size_t adapter_workspace(int64_t tokens, int64_t rank, int64_t adapters);
cudaError_t adapter_forward_launch(const AdapterDesc& d, int num_sms, cudaStream_t stream, std::string* why);
cudaError_t adapter_backward_launch(const AdapterDesc& d, int num_sms, cudaStream_t stream, std::string* why);

}  // namespace tl

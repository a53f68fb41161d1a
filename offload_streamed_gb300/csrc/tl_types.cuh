// tl_types.cuh -- 16-byte vectors of the element types that the operators
// around the product take (bf16, fp16, fp32), to and from fp32.
#pragma once
#include "tiled_linear.h"

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tl {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}

// N elements that are loaded and stored as one access (N = 16 bytes' worth),
// or a single element (N = 1).
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
    T v[N];
};

// Element i of an array whose type is known at run time.
__device__ __forceinline__ float load_as_f32(const void* p, int32_t type, int64_t i) {
    if (type == TL_TYPE_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
    if (type == TL_TYPE_F16) return to_f32(static_cast<const __half*>(p)[i]);
    return static_cast<const float*>(p)[i];
}

inline size_t type_bytes(int32_t type) { return type == TL_TYPE_F32 ? 4 : 2; }
inline bool type_known(int32_t type) { return type >= TL_TYPE_BF16 && type <= TL_TYPE_F32; }

}  // namespace tl

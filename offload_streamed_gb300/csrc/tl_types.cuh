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

// Two fp32 values that go through one instruction (add, multiply and fused
// multiply-add of register pairs), or one.  Which of them a kernel holds
// depends on its vectors: Lanes<N> is the type, kLanes its count.
__device__ __forceinline__ uint64_t bits2(float2 v) {
    uint64_t b;
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(v.x), "f"(v.y));
    return b;
}
__device__ __forceinline__ float2 pair2(uint64_t b) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(b));
    return v;
}
__device__ __forceinline__ float2 add(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(r);
}
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ float total(float2 v) { return v.x + v.y; }
__device__ __forceinline__ float total(float v) { return v; }

template <int N>
struct LanesOf {
    using type = float2;
};
template <>
struct LanesOf<1> {
    using type = float;
};
template <int N>
using Lanes = typename LanesOf<N>::type;

template <typename L>
__device__ __forceinline__ L splat(float v);
template <>
__device__ __forceinline__ float2 splat<float2>(float v) {
    return make_float2(v, v);
}
template <>
__device__ __forceinline__ float splat<float>(float v) {
    return v;
}

// A vector as fp32 lanes, and back (rounded to nearest even).
template <typename T>
__device__ __forceinline__ void unpack(const Vec<T, 1>& u, float (&v)[1]) {
    v[0] = to_f32(u.v[0]);
}
__device__ __forceinline__ void unpack(const Vec<float, 4>& u, float2 (&v)[2]) {
    v[0] = make_float2(u.v[0], u.v[1]);
    v[1] = make_float2(u.v[2], u.v[3]);
}
__device__ __forceinline__ void unpack(const Vec<__half, 8>& u, float2 (&v)[4]) {
    const __half2* h = reinterpret_cast<const __half2*>(u.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(h[i]);
}
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, 8>& u, float2 (&v)[4]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u.v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void pack(const float (&v)[1], Vec<T, 1>& u) {
    u.v[0] = from_f32<T>(v[0]);
}
__device__ __forceinline__ void pack(const float2 (&v)[2], Vec<float, 4>& u) {
    u.v[0] = v[0].x;
    u.v[1] = v[0].y;
    u.v[2] = v[1].x;
    u.v[3] = v[1].y;
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Vec<__half, 8>& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<__half2*>(u.v)[i] = __float22half2_rn(v[i]);
}
__device__ __forceinline__ void pack(const float2 (&v)[4], Vec<__nv_bfloat16, 8>& u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<__nv_bfloat162*>(u.v)[i] = __float22bfloat162_rn(v[i]);
}

// Four of them from element i on, which is a multiple of four, the array's start
// being 16-byte aligned.
__device__ __forceinline__ Vec<float, 4> load4_as_f32(const void* p, int32_t type, int64_t i) {
    if (type == TL_TYPE_F32) return *reinterpret_cast<const Vec<float, 4>*>(static_cast<const float*>(p) + i);
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    Vec<float, 4> v;
    if (type == TL_TYPE_BF16) {
        v.v[0] = __uint_as_float(u.x << 16);
        v.v[1] = __uint_as_float(u.x & 0xffff0000u);
        v.v[2] = __uint_as_float(u.y << 16);
        v.v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        v.v[0] = a.x;
        v.v[1] = a.y;
        v.v[2] = b.x;
        v.v[3] = b.y;
    }
    return v;
}

inline size_t type_bytes(int32_t type) { return type == TL_TYPE_F32 ? 4 : 2; }
inline bool type_known(int32_t type) { return type >= TL_TYPE_BF16 && type <= TL_TYPE_F32; }

}  // namespace tl

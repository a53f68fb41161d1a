// tl_fp8_quant.cu -- matrices to 8-bit floating point with a power-of-two
// scale for each block of 128.
//
//   scale = 2^e, e the least whole number with amax <= top * 2^e
//   q     = round(x / scale) to e4m3 (top = 448) or e5m2 (top = 57344)
//
// A block is 128 elements of a row, 128 of a column, or 128 x 128; the three
// forms serve the two operands of a linear layer's three products.  Dividing by
// a power of two is exact, so each element is rounded once.  A block of zeros
// has scale 1; a block with an infinity or a NaN has the NaN scale (byte 255),
// and so makes NaN of every result that it enters.
//
// Bound by memory: two bytes read and one written for an element and form.  A
// CTA takes a 128 x 128 tile, each thread eight 8-element pieces of rows, and
// keeps it in registers: every form that is wanted comes from one reading.
#include "tl_fp8.h"
#include "tl_types.cuh"

#include <cuda_fp8.h>

namespace tl {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPer = 8;  // rows of a thread, 16 apart

struct QuantArgs {
    const void* x;
    int64_t ldx;
    int64_t rows, cols;
    Fp8QuantDesc::Form row, col, tile;
    int32_t emax;  // exponent of the format's largest power of two
    int32_t vec_in;
};

// The scale's byte for a block's largest magnitude (NaN: not finite).
__device__ __forceinline__ uint32_t scale_byte(float amax, int emax) {
    const uint32_t b = __float_as_uint(amax);
    if (b == 0) return 127;
    if (b >= 0x7f800000u) return 255;
    // amax = m 2^p: the format's top is 1.75 * 2^emax
    const int e = int(b >> 23) - 127 - emax + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return uint32_t(max(e, -127) + 127);
}
// 2^-(byte - 127); 0 for the NaN scale, whose values do not matter
__device__ __forceinline__ float unscale(uint32_t byte) {
    if (byte == 255) return 0.0f;
    return byte == 254 ? __uint_as_float(1u << 22) : __uint_as_float((254u - byte) << 23);
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
    constexpr __nv_fp8_interpretation_t f = E5M2 ? __NV_E5M2 : __NV_E4M3;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, f);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, f);
    return lo | (hi << 16);
}

__device__ __forceinline__ void store8(const Fp8QuantDesc::Form& f, int64_t r, int64_t c, int64_t cols, uint32_t lo,
                                       uint32_t hi) {
    uint8_t* dst = f.q + r * f.ldq + c;
    if (c + 8 <= cols && (reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) dst[i] = uint8_t((i < 4 ? lo >> (8 * i) : hi >> (8 * i - 32)) & 255u);
    }
}

template <typename T, bool E5M2>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const QuantArgs p) {
    __shared__ float part[16][kFp8Block];  // column maxima of the 16 threads that share a column
    __shared__ float warp_max[kThreads / 32];
    const int lane16 = threadIdx.x & 15, r16 = threadIdx.x >> 4;
    const int64_t c0 = int64_t(blockIdx.x) * kFp8Block, c = c0 + lane16 * 8;
    const int64_t r0 = int64_t(blockIdx.y) * kFp8Block;
    float v[kRowsPer][8];
    const T* x = static_cast<const T*>(p.x);
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
        const int64_t r = r0 + r16 + 16 * k;
        if (r < p.rows && p.vec_in && c + 8 <= p.cols) {
            constexpr int N = 16 / sizeof(T);
            const Vec<T, N>* src = reinterpret_cast<const Vec<T, N>*>(x + r * p.ldx + c);
#pragma unroll
            for (int q = 0; q < 8 / N; ++q) {
                const Vec<T, N> u = src[q];
#pragma unroll
                for (int i = 0; i < N; ++i) v[k][q * N + i] = to_f32(u.v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = r < p.rows && c + i < p.cols ? to_f32(x[r * p.ldx + c + i]) : 0.0f;
        }
    }
    // rows: the 16 threads of a row are half a warp
    float all = 0;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
        float m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[k][i]));
        all = max_nan(all, m);
        if (!p.row.q) continue;
#pragma unroll
        for (int s = 8; s; s >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, s));
        const int64_t r = r0 + r16 + 16 * k;
        const uint32_t byte = scale_byte(m, p.emax);
        const float f = unscale(byte);
        if (r < p.rows) {
            store8(p.row, r, c, p.cols, quant4<E5M2>(v[k][0] * f, v[k][1] * f, v[k][2] * f, v[k][3] * f),
                   quant4<E5M2>(v[k][4] * f, v[k][5] * f, v[k][6] * f, v[k][7] * f));
            if (lane16 == 0) p.row.scale[r * p.row.lds + blockIdx.x] = uint8_t(byte);
        }
    }
    if (p.tile.q) {
        all = max_nan(all, __shfl_xor_sync(~0u, all, 16));
#pragma unroll
        for (int s = 8; s; s >>= 1) all = max_nan(all, __shfl_xor_sync(~0u, all, s));
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = all;
        __syncthreads();
        float m = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max_nan(m, warp_max[w]);
        const uint32_t byte = scale_byte(m, p.emax);
        const float f = unscale(byte);
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) {
            const int64_t r = r0 + r16 + 16 * k;
            if (r < p.rows)
                store8(p.tile, r, c, p.cols, quant4<E5M2>(v[k][0] * f, v[k][1] * f, v[k][2] * f, v[k][3] * f),
                       quant4<E5M2>(v[k][4] * f, v[k][5] * f, v[k][6] * f, v[k][7] * f));
        }
        if (threadIdx.x == 0) p.tile.scale[int64_t(blockIdx.y) * p.tile.lds + blockIdx.x] = uint8_t(byte);
    }
    if (p.col.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float m = 0;
#pragma unroll
            for (int k = 0; k < kRowsPer; ++k) m = max_nan(m, fabsf(v[k][i]));
            part[r16][lane16 * 8 + i] = m;
        }
        __syncthreads();
        if (threadIdx.x < kFp8Block) {
            float m = 0;
#pragma unroll
            for (int w = 0; w < 16; ++w) m = max_nan(m, part[w][threadIdx.x]);
            const uint32_t byte = scale_byte(m, p.emax);
            part[0][threadIdx.x] = unscale(byte);
            if (c0 + threadIdx.x < p.cols) p.col.scale[int64_t(blockIdx.y) * p.col.lds + c0 + threadIdx.x] = uint8_t(byte);
        }
        __syncthreads();
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = part[0][lane16 * 8 + i];
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) {
            const int64_t r = r0 + r16 + 16 * k;
            if (r < p.rows)
                store8(p.col, r, c, p.cols, quant4<E5M2>(v[k][0] * f[0], v[k][1] * f[1], v[k][2] * f[2], v[k][3] * f[3]),
                       quant4<E5M2>(v[k][4] * f[4], v[k][5] * f[5], v[k][6] * f[6], v[k][7] * f[7]));
        }
    }
}

template <typename T>
void launch(const QuantArgs& a, bool e5m2, dim3 grid, cudaStream_t stream) {
    if (e5m2) fp8_quantize_kernel<T, true><<<grid, kThreads, 0, stream>>>(a);
    else fp8_quantize_kernel<T, false><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

std::string fp8_quantize_check(const Fp8QuantDesc& d) {
    if (d.rows < 0 || d.cols < 1) return "rows must be >= 0 and cols >= 1";
    if (d.rows > int64_t(65535) * kFp8Block || d.cols > (int64_t(1) << 30)) return "matrix too large";
    if (!type_known(d.type)) return "unknown tl_type";
    if (d.format != TL_FP8_E4M3 && d.format != TL_FP8_E5M2) return "unknown tl_fp8_format";
    if (d.rows == 0) return {};
    if (!d.row.q && !d.col.q && !d.tile.q) return "no form is wanted";
    if (!d.x || reinterpret_cast<uintptr_t>(d.x) % type_bytes(d.type)) return "x is null or not aligned to its type";
    if (d.ldx < d.cols) return "the leading dimension of x is smaller than cols";
    const int64_t cb = (d.cols + kFp8Block - 1) / kFp8Block;
    for (const auto& f : {d.row, d.col, d.tile})
        if (f.q && (!f.scale || f.ldq < d.cols)) return "a form has no scales, or a leading dimension smaller than cols";
    if ((d.row.q && d.row.lds < cb) || (d.col.q && d.col.lds < d.cols) || (d.tile.q && d.tile.lds < cb))
        return "a leading dimension of scales is too small";
    return {};
}

cudaError_t fp8_quantize_launch(const Fp8QuantDesc& d, cudaStream_t stream) {
    if (d.rows == 0) return cudaSuccess;
    QuantArgs a{};
    a.x = d.x;
    a.ldx = d.ldx;
    a.rows = d.rows;
    a.cols = d.cols;
    a.row = d.row;
    a.col = d.col;
    a.tile = d.tile;
    const bool e5m2 = d.format == TL_FP8_E5M2;
    a.emax = e5m2 ? 15 : 8;
    const int64_t vec = int64_t(16 / type_bytes(d.type));
    a.vec_in = (reinterpret_cast<uintptr_t>(d.x) & 15) == 0 && d.ldx % vec == 0;
    const dim3 grid(unsigned((d.cols + kFp8Block - 1) / kFp8Block), unsigned((d.rows + kFp8Block - 1) / kFp8Block));
    if (d.type == TL_TYPE_BF16) launch<__nv_bfloat16>(a, e5m2, grid, stream);
    else if (d.type == TL_TYPE_F16) launch<__half>(a, e5m2, grid, stream);
    else launch<float>(a, e5m2, grid, stream);
    return cudaGetLastError();
}

}  // namespace tl

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
    int32_t vec;   // rows of x start on 16-byte boundaries, rows of the results on 8-byte ones
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

// The scale of block b of `blocks` of vector i of n: a byte of the word
// [b / 4][i]; the last block writes the bytes that follow it, too.
__device__ __forceinline__ void store_scale(uint8_t* scale, uint32_t b, uint32_t blocks, int64_t i, int64_t n, uint32_t byte) {
    uint8_t* word = scale + (int64_t(b / 4) * n + i) * 4;
    word[b % 4] = uint8_t(byte);
    if (b == blocks - 1)
        for (uint32_t j = b % 4 + 1; j < 4; ++j) word[j] = 127;
}

// Eight elements of a row as they were read, and what is done with them.
template <typename T>
struct Eight {
    static constexpr int N = 16 / sizeof(T), kVecs = 8 / N;
    Vec<T, N> u[kVecs];
    __device__ __forceinline__ float at(int i) const { return to_f32(u[i / N].v[i % N]); }
};
// The largest magnitude; a NaN stays.  16-bit types in pairs.
__device__ __forceinline__ float amax8(const Eight<float>& e) {
    float m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(e.at(i)));
    return m;
}
__device__ __forceinline__ float amax8(const Eight<__half>& e) {
    const __half2* h = reinterpret_cast<const __half2*>(e.u[0].v);
    const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}
__device__ __forceinline__ float amax8(const Eight<__nv_bfloat16>& e) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(e.u[0].v);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
}

// FORMS: which of the forms are made (bit 0 rows, 1 columns, 2 tiles).
// WHOLE: the tile lies inside the matrix, on 16-byte (values) and 8-byte
// (results) boundaries, so that nothing is asked of its elements.
template <typename T, bool E5M2, int FORMS, bool WHOLE>
__device__ __forceinline__ void quantize_tile(const QuantArgs& p, float (*part)[kFp8Block], float* warp_max) {
    const int lane16 = threadIdx.x & 15, r16 = threadIdx.x >> 4;
    const int64_t c0 = int64_t(blockIdx.x) * kFp8Block, c = c0 + lane16 * 8;
    const int64_t r0 = int64_t(blockIdx.y) * kFp8Block;
    Eight<T> v[kRowsPer];
    const T* x = static_cast<const T*>(p.x) + (r0 + r16) * p.ldx + c;
#pragma unroll
    for (int k = 0; k < kRowsPer; ++k) {
        const T* src = x + int64_t(16 * k) * p.ldx;
        if constexpr (WHOLE) {
#pragma unroll
            for (int q = 0; q < Eight<T>::kVecs; ++q)
                v[k].u[q] = reinterpret_cast<const Vec<T, Eight<T>::N>*>(src)[q];
        } else {
            const bool in = r0 + r16 + 16 * k < p.rows;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k].u[i / Eight<T>::N].v[i % Eight<T>::N] = in && c + i < p.cols ? src[i] : from_f32<T>(0.0f);
        }
    }
    // write a row's eight, each times the power of two for its column
    auto store = [&](const Fp8QuantDesc::Form& f, int k, const float (&by)[8]) {
        const int64_t r = r0 + r16 + 16 * k;
        const uint32_t lo = quant4<E5M2>(v[k].at(0) * by[0], v[k].at(1) * by[1], v[k].at(2) * by[2], v[k].at(3) * by[3]);
        const uint32_t hi = quant4<E5M2>(v[k].at(4) * by[4], v[k].at(5) * by[5], v[k].at(6) * by[6], v[k].at(7) * by[7]);
        uint8_t* dst = f.q + r * f.ldq + c;
        if constexpr (WHOLE) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else if (r < p.rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < p.cols) dst[i] = uint8_t((i < 4 ? lo >> (8 * i) : hi >> (8 * i - 32)) & 255u);
        }
    };
    auto all8 = [](float f, float (&by)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) by[i] = f;
    };
    float m[kRowsPer], by[8];
    if constexpr ((FORMS & 5) != 0) {
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) m[k] = amax8(v[k]);
    }
    if constexpr ((FORMS & 4) != 0) {
        float all = m[0];
#pragma unroll
        for (int k = 1; k < kRowsPer; ++k) all = max_nan(all, m[k]);
#pragma unroll
        for (int s = 16; s; s >>= 1) all = max_nan(all, __shfl_xor_sync(~0u, all, s));
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = all;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) all = max_nan(all, warp_max[w]);
        const uint32_t byte = scale_byte(all, p.emax);
        all8(unscale(byte), by);
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) store(p.tile, k, by);
        if (threadIdx.x == 0) p.tile.scale[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = uint8_t(byte);
    }
    if constexpr ((FORMS & 1) != 0) {  // the 16 threads of a row are half a warp
#pragma unroll
        for (int s = 8; s; s >>= 1)
#pragma unroll
            for (int k = 0; k < kRowsPer; ++k) m[k] = max_nan(m[k], __shfl_xor_sync(~0u, m[k], s));
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) {
            const int64_t r = r0 + r16 + 16 * k;
            const uint32_t byte = scale_byte(m[k], p.emax);
            all8(unscale(byte), by);
            store(p.row, k, by);
            if (lane16 == 0 && (WHOLE || r < p.rows)) store_scale(p.row.scale, blockIdx.x, gridDim.x, r, p.rows, byte);
        }
    }
    if constexpr ((FORMS & 2) != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float mc = fabsf(v[0].at(i));
#pragma unroll
            for (int k = 1; k < kRowsPer; ++k) mc = max_nan(mc, fabsf(v[k].at(i)));
            by[i] = max_nan(mc, __shfl_xor_sync(~0u, mc, 16));  // the two rows of a warp
        }
        if ((threadIdx.x & 31) < 16) {
            float4* dst = reinterpret_cast<float4*>(&part[threadIdx.x >> 5][lane16 * 8]);
            dst[0] = make_float4(by[0], by[1], by[2], by[3]);
            dst[1] = make_float4(by[4], by[5], by[6], by[7]);
        }
        __syncthreads();
        if (threadIdx.x < kFp8Block) {
            float mc = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) mc = max_nan(mc, part[w][threadIdx.x]);
            const uint32_t byte = scale_byte(mc, p.emax);
            part[0][threadIdx.x] = unscale(byte);
            if (c0 + threadIdx.x < p.cols) store_scale(p.col.scale, blockIdx.y, gridDim.y, c0 + threadIdx.x, p.cols, byte);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) by[i] = part[0][lane16 * 8 + i];
#pragma unroll
        for (int k = 0; k < kRowsPer; ++k) store(p.col, k, by);
    }
}

template <typename T, bool E5M2, int FORMS>
__global__ void __launch_bounds__(kThreads, 3) fp8_quantize_kernel(const QuantArgs p) {
    __shared__ __align__(16) float part[kThreads / 32][kFp8Block];  // column maxima, by warp
    __shared__ float warp_max[kThreads / 32];
    // a product that was launched to begin early may: it waits for this kernel
    // before it reads what is written here
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool whole = p.vec && int64_t(blockIdx.x + 1) * kFp8Block <= p.cols && int64_t(blockIdx.y + 1) * kFp8Block <= p.rows;
    if (whole) quantize_tile<T, E5M2, FORMS, true>(p, part, warp_max);
    else quantize_tile<T, E5M2, FORMS, false>(p, part, warp_max);
}

template <typename T, bool E5M2>
void launch(const QuantArgs& a, int forms, dim3 grid, cudaStream_t stream) {
    switch (forms) {
        case 1: fp8_quantize_kernel<T, E5M2, 1><<<grid, kThreads, 0, stream>>>(a); break;
        case 2: fp8_quantize_kernel<T, E5M2, 2><<<grid, kThreads, 0, stream>>>(a); break;
        case 3: fp8_quantize_kernel<T, E5M2, 3><<<grid, kThreads, 0, stream>>>(a); break;
        case 4: fp8_quantize_kernel<T, E5M2, 4><<<grid, kThreads, 0, stream>>>(a); break;
        case 5: fp8_quantize_kernel<T, E5M2, 5><<<grid, kThreads, 0, stream>>>(a); break;
        case 6: fp8_quantize_kernel<T, E5M2, 6><<<grid, kThreads, 0, stream>>>(a); break;
        default: fp8_quantize_kernel<T, E5M2, 7><<<grid, kThreads, 0, stream>>>(a); break;
    }
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
    for (const auto& f : {d.row, d.col, d.tile})
        if (f.q && (!f.scale || f.ldq < d.cols)) return "a form has no scales, or a leading dimension smaller than cols";
    for (const auto& f : {d.row, d.col})
        if (f.q && (reinterpret_cast<uintptr_t>(f.scale) & 3)) return "scales of the row and col forms must be 4-byte aligned";
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
    a.vec = (reinterpret_cast<uintptr_t>(d.x) & 15) == 0 && d.ldx % vec == 0;
    int forms = 0, bit = 1;
    for (const auto* f : {&d.row, &d.col, &d.tile}) {
        if (f->q) {
            forms |= bit;
            a.vec = a.vec && (reinterpret_cast<uintptr_t>(f->q) & 7) == 0 && f->ldq % 8 == 0;
        }
        bit *= 2;
    }
    const dim3 grid(unsigned((d.cols + kFp8Block - 1) / kFp8Block), unsigned((d.rows + kFp8Block - 1) / kFp8Block));
    auto run = [&](auto zero) {
        using T = decltype(zero);
        if (e5m2) launch<T, true>(a, forms, grid, stream);
        else launch<T, false>(a, forms, grid, stream);
    };
    if (d.type == TL_TYPE_BF16) run(__nv_bfloat16{});
    else if (d.type == TL_TYPE_F16) run(__half{});
    else run(float{});
    return cudaGetLastError();
}

}  // namespace tl

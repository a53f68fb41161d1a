// tl_fp8.h -- internal interface of the 8-bit products (host side).
//
// A matrix in 8 bits is its values (e4m3 or e5m2, one byte each) and, for each
// block of 128, a scale 2^(byte - 127).  The blocks run along the reduction:
// of an operand's 128 reduction indices at one of its other indices ("vector"
// scales), or at 128 of them ("block" scales, the weight's).
#pragma once
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

namespace tl {

constexpr int kFp8Block = 128;

// Quantise x [rows, cols]: up to three forms from one reading of it.
struct Fp8QuantDesc {
    int64_t rows = 0, cols = 0;
    int32_t type = 0;  // tl_type of x
    const void* x = nullptr;
    int64_t ldx = 0;
    int32_t format = 0;  // tl_fp8_format
    struct Form {
        uint8_t* q = nullptr;  // [rows, cols], ld ldq; nullptr: not wanted
        int64_t ldq = 0;
        uint8_t* scale = nullptr;
    } row, col, tile;  // scales [cols/512][rows][4], [rows/512][cols][4], [rows/128][cols/128]
};
std::string fp8_quantize_check(const Fp8QuantDesc& d);
cudaError_t fp8_quantize_launch(const Fp8QuantDesc& d, cudaStream_t stream);

// One operand of a product: element (i, k), i its own index (a row of the
// result for A, a column for B), k the reduction's.
struct Fp8Operand {
    const void* q = nullptr;
    int64_t ld = 0;
    bool mn_major = false;  // (i, k) at q[k * ld + i]; else at q[i * ld + k]
    int32_t format = 0;
    // Vectors: byte k / 128 % 4 of the word [k / 512][i].  Tiles: byte
    // [i / 128][k / 128] or, where the reduction runs down the rows (mn_major),
    // [k / 128][i / 128] of a matrix of tile_cols columns.
    const void* scale = nullptr;
    bool tiles = false;
    int64_t tile_cols = 0;
};
// D [m, n] (bf16, ld ldd) = sum over k of A (i, k) B (j, k)
struct Fp8GemmDesc {
    int64_t m_dim = 0, n_dim = 0, k_dim = 0;
    Fp8Operand a, b;
    void* d = nullptr;
    int64_t ldd = 0;
    int32_t* err = nullptr;
    // The kernel before this one in the stream writes A alone: B may be read
    // before that kernel has completed.
    bool early = false;
};
std::string fp8_gemm_check(const Fp8GemmDesc& g);
cudaError_t fp8_gemm_launch(const Fp8GemmDesc& g, int num_sms, cudaStream_t stream, std::string* why);

}  // namespace tl

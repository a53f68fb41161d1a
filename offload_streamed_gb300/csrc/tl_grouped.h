// tl_grouped.h -- internal interface of the products whose weight depends on the
// row (host side): rows p = 0 .. rows - 1 in an order in which group g owns
// offsets[g] .. offsets[g + 1] - 1, and a weight for each group.
#pragma once
#include <cstdint>
#include <string>
#include <cuda_runtime.h>

namespace tl {

// A matrix whose row for place p is index[p] (p itself without an index).
struct RowsOperand {
    const void* at = nullptr;
    int64_t ld = 0;
    int64_t count = 0;  // rows of the matrix
    const int32_t* index = nullptr;
};

// Indexed rows sorted into a matrix [rows, cols] of 16-bit elements, ld picked_ld.
int64_t picked_ld(int64_t cols);
cudaError_t pick_rows_launch(const RowsOperand& x, int64_t rows, int64_t cols, void* out, cudaStream_t stream);

// out[row(p), own] = scale[g] sum_k x[row(p), k] w[g](k, own)
struct GroupedDesc {
    int64_t rows = 0, reduce = 0, own = 0, groups = 0;
    int32_t type = 0;  // TL_TYPE_BF16 or TL_TYPE_F16, of x, w and out
    const int32_t* offsets = nullptr;
    RowsOperand x;
    const void* w = nullptr;
    int64_t ldw = 0, w_apart = 0;
    bool own_contiguous = true;  // w[g] is [reduce, own]; else [own, reduce]
    RowsOperand out;                // at is written
    // From here on for own <= 128 (as an indexed out).  all_rows: rows behind the last group are written, too, as zeros.
    bool all_rows = false;
    const float* scale = nullptr;  // [groups]; nullptr: scale_all
    float scale_all = 1.0f;
    // Not nullptr (own <= 128): the unrounded result, too, as two parts of split_half
    // columns whose sum it is to twice the type's digits; [rows, 2 split_half], by place.
    // fp16's parts are of the result in units of split_units[place], a power of two.
    void* split_out = nullptr;
    int32_t split_half = 0;
    float* split_units = nullptr;  // [rows], by place; fp16 only
    void* gathered = nullptr;  // workspace for an indexed x's rows, [rows, picked_ld] (own > 128 needs it)
    int32_t* err = nullptr;
};
std::string grouped_check(const GroupedDesc& d);
cudaError_t grouped_launch(const GroupedDesc& d, int num_sms, cudaStream_t stream, std::string* why);

// dw[g](i, j) = scale[g] sum over g's places of x[row(p), i] dy[row(p), j]
struct GroupedDwDesc {
    int64_t rows = 0, m_dim = 0, n_dim = 0, groups = 0;
    int32_t type = 0;
    const int32_t* offsets = nullptr;
    RowsOperand x, dy;
    int32_t half = 0;  // not 0: dy's columns are two parts of `half`, which are added (n_dim <= half)
    const float* dy_units = nullptr;  // [rows], by place: what dy's two parts are in units of, powers of two; nullptr: ones
    void* dw = nullptr;
    int64_t lddw = 0, dw_apart = 0;
    void* gathered = nullptr;  // workspace for an indexed x's rows, [rows, picked_ld] (n_dim > 128 needs it)
    bool transposed = false;  // dw[g] is [n_dim, m_dim] (n_dim <= 128 only)
    const float* scale = nullptr;
    float scale_all = 1.0f;
    int32_t* err = nullptr;
};
std::string grouped_dw_check(const GroupedDwDesc& d);
cudaError_t grouped_dw_launch(const GroupedDwDesc& d, int num_sms, cudaStream_t stream, std::string* why);

}  // namespace tl

// tl_err_word.h -- internal interface of the operators' own error word (host side).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace tl {

// The address of the current device's word.
cudaError_t operator_err_word(int32_t** out);

}  // namespace tl

// tl_err_word.cu -- an error word of each device for the operators around the
// product, for callers that have none of their own.  It is a variable of the
// library's, zero when it is loaded: nothing is allocated and no copy or wait is
// enqueued for it, so a call's first use of it may stand in a stream capture.
#include "tl_err_word.h"

namespace tl {
namespace {
__device__ int32_t g_operator_err = 0;
}

cudaError_t operator_err_word(int32_t** out) {
    // Loading the library's code on a device may allocate there, which a capture
    // that runs in this thread would refuse.
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_operator_err);
    cudaThreadExchangeStreamCaptureMode(&mode);
    *out = static_cast<int32_t*>(p);
    return e;
}

}  // namespace tl

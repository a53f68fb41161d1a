// tl_entry.h -- what the operators' C entry points share: refusals with a message,
// and nothing thrown across the ABI.
#pragma once
#include "tiled_linear.h"
#include "tl_unbound_error.h"

#include <cstdint>
#include <cuda_runtime.h>
#include <exception>
#include <string>

namespace tl {

inline tl_status refuse(tl_status st, const std::string& why) {
    set_unbound_error(why);
    return st;
}

inline tl_status done(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return TL_OK;
    return refuse(TL_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

// Nothing is thrown across the ABI.
template <typename F>
tl_status guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception& e) {
        return refuse(TL_ERR_STATE, e.what());
    } catch (...) {
        return refuse(TL_ERR_STATE, "unknown exception");
    }
}

inline bool workspace_ok(const void* p, size_t have, size_t need) {
    return p && (reinterpret_cast<uintptr_t>(p) & 255u) == 0 && have >= need;
}

}  // namespace tl

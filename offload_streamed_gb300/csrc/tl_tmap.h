// tl_tmap.h -- tensor maps of the operators' kernels: row-major matrices (and
// stacks of them) read or written in boxes of 128-byte rows, 128B-swizzled.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <string>

namespace tl {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// `count` matrices (`apart` elements from one to the next) of `outer` rows of
// `inner` elements, rows `ld` elements apart; boxes of 128 bytes x box_outer
// rows.  Zero fill outside (loads), clipping (stores).
inline bool swizzled_map(CUtensorMap* map, CUtensorMapDataType type, uint32_t esize, const void* base, uint64_t inner,
                         uint64_t outer, uint64_t ld, uint32_t box_outer, std::string* why, uint64_t count = 1,
                         uint64_t apart = 0) {
    auto fn = tensor_map_encoder();
    if (!fn) {
        if (why) *why = "cuTensorMapEncodeTiled is unavailable from the driver";
        return false;
    }
    const bool stack = apart != 0;
    cuuint64_t dims[3] = {inner, outer, count};
    cuuint64_t strides[2] = {ld * esize, apart * esize};
    cuuint32_t box[3] = {128 / esize, box_outer, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, type, stack ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        if (why) *why = "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(int(r));
        return false;
    }
    return true;
}

}  // namespace tl

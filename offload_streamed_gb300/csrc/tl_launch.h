// tl_launch.h -- what the host asks the runtime about a kernel or a device,
// asked once: the answers depend on the kernel, its launch shape and the
// device alone, and asking again would cost a small call more than its launch.
#pragma once
#include <cuda_runtime.h>

#include <map>
#include <mutex>
#include <tuple>

namespace tl {

// CTAs of the kernel that an SM of the current device holds, with `smem` bytes
// of dynamic shared memory each (which the kernel is allowed here).
inline cudaError_t ctas_per_sm(const void* kernel, int threads, size_t smem, int* out) {
    static std::mutex lock;
    static std::map<std::tuple<int, const void*, int, size_t>, int> known;
    static std::map<std::pair<int, const void*>, size_t> allowed;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> hold(lock);
    const auto key = std::make_tuple(dev, kernel, threads, smem);
    const auto it = known.find(key);
    if (it != known.end()) {
        *out = it->second;
        return cudaSuccess;
    }
    size_t& most = allowed[{dev, kernel}];  // never lowered: an earlier shape may need it
    if (smem > most) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        most = smem;
    }
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, kernel, threads, smem);
    if (e == cudaSuccess) known[key] = *out;
    return e;
}

// Clusters of `cluster` CTAs of the kernel that the current device runs at a
// time.  A cluster stays within one GPC, so there may be fewer than the SMs'
// CTAs would make; a grid of more is run in turns.  Call ctas_per_sm first,
// which allows the kernel its shared memory.
inline cudaError_t clusters_at_a_time(const void* kernel, int threads, size_t smem, int cluster, int* out) {
    static std::mutex lock;
    static std::map<std::tuple<int, const void*, int, size_t, int>, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> hold(lock);
    const auto key = std::make_tuple(dev, kernel, threads, smem, cluster);
    const auto it = known.find(key);
    if (it != known.end()) {
        *out = it->second;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(cluster));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(out, kernel, &cfg);
    if (e == cudaSuccess) known[key] = *out;
    return e;
}

// SMs of the current device; 0 if it cannot be told.
inline int device_sms() {
    static std::mutex lock;
    static std::map<int, int> known;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> hold(lock);
    const auto it = known.find(dev);
    if (it != known.end()) return it->second;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    known[dev] = sms;
    return sms;
}

}  // namespace tl

// launch_util.h -- host-side helpers shared by the kernel launchers.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace rfx {

// A kernel's dynamic shared-memory limit, raised to at least `bytes` on the
// current device the first time a launch needs it.  Thread-safe: a lock-free
// check on the fast path, the attribute set under a lock, and the recorded
// limit only grows (so a smaller request never lowers a larger one).  Not a
// stream operation, so it stays out of graph captures after the first call.
class SmemLimit {
  public:
    cudaError_t ensure(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool cached = dev >= 0 && dev < kDevices;
        if (cached && set_[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
        std::lock_guard<std::mutex> guard(mu_);
        if (cached && set_[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && cached) set_[dev].store(bytes, std::memory_order_release);
        return e;
    }

  private:
    static constexpr int kDevices = 64;
    std::atomic<int> set_[kDevices] = {};
    std::mutex mu_;
};

// SM count of the current device, queried once per device.
inline cudaError_t device_sms(int& sms) {
    static std::atomic<int> cache[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < 64;
    if (cached && (sms = cache[dev].load(std::memory_order_relaxed)) != 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && cached) cache[dev].store(sms, std::memory_order_relaxed);
    return e;
}

// How many clusters of `size` (at most 8) CTAs of a kernel run on the current device at once, asked once per
// kernel (an object each), device and size.
class ClusterFit {
  public:
    template <typename... Params>
    cudaError_t get(void (*kernel)(Params...), int size, unsigned block, size_t smem, int& clusters) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool cached = dev >= 0 && dev < kDevices;
        if (cached && (clusters = fit_[dev][size].load(std::memory_order_relaxed) - 1) >= 0) return cudaSuccess;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(block);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = size;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
        if (e == cudaSuccess && cached) fit_[dev][size].store(clusters + 1, std::memory_order_relaxed);
        return e;
    }

  private:
    static constexpr int kDevices = 64;
    std::atomic<int> fit_[kDevices][9] = {};
};

// Launch as a programmatic dependent of the kernel before it on the stream:
// the launch overlaps that kernel's tail, and the kernel itself waits
// (grid_dep_wait) before its first access to global memory.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    (void)cudaGetLastError();   // an earlier call's launch error is not this launch's
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The same in clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), unsigned grid, unsigned cluster, unsigned block, size_t smem,
                            cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    (void)cudaGetLastError();   // an earlier call's launch error is not this launch's
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace rfx

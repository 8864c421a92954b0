// ce_launch.h -- what the launchers of ce_objectives.cu, ce_choices.cu and ce_router.cu share:
// a launch's configuration, a kernel's attributes, and the devices on which a
// file's kernels have been launched.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "ce_internal.h"

namespace cerows {

// cluster 0: a launch without cluster dimensions, for kernels that execute no
// instruction on shared::cluster addresses (st.async is illegal there, to the
// CTA's own shared memory too).
struct LaunchConfig {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    LaunchConfig(int64_t ctas, int threads, int cluster, bool dependent, cudaStream_t s, int smem = 0) {
        cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
        cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.stream = s;
        int n = 0;
        if (cluster > 0) {
            attr[n].id = cudaLaunchAttributeClusterDimension;
            attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
            ++n;
        }
        if (dependent) {
            attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[n].val.programmaticStreamSerializationAllowed = 1;
            ++n;
        }
        cfg.attrs = attr;
        cfg.numAttrs = n;
    }
};

static_assert(kMaxDevices <= 64, "a bit per device");
inline uint64_t bit_of(const DeviceInfo &dev) { return uint64_t(1) << dev.device; }

// Devices (a bit each) that have launched a kernel of a file. Touching a kernel
// or a variable of a file loads all of its code, 10 ms once: no function of the
// library's does so for another file's.
class Launches {
    std::atomic<uint64_t> on_{0};

  public:
    bool any(const DeviceInfo &dev) const { return on_.load(std::memory_order_acquire) & bit_of(dev); }
    void note(const DeviceInfo &dev) {
        if (!any(dev)) on_.fetch_or(bit_of(dev), std::memory_order_release);
    }
};

// A kernel and the devices on which its attributes are set: clusters of up to 16
// CTAs, and as much shared memory as a CTA may have. Set at the kernel's first
// launch on a device.
struct Kernel {
    const void *fn;
    bool smem;
    std::atomic<uint64_t> set{0};
    Kernel(const void *f, bool dynamic_smem) : fn(f), smem(dynamic_smem) {}
};
inline cudaError_t ready(Kernel &k, const DeviceInfo &dev) {
    const uint64_t bit = bit_of(dev);
    if (k.set.load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && k.smem)
        e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, dev.max_smem_optin);
    if (e == cudaSuccess) k.set.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace cerows

// Host: a kernel's opt-in to more dynamic shared memory than 48 KB.
//
// The attribute belongs to the device that is current when it is set, not to the process: a kernel that was opted
// in on one device does not launch on the next.  One object stands beside each kernel; a call on a device that it
// knows costs a look-up.
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

#include <atomic>

namespace pa {

class SmemOptIn {
public:
    // Lets `kern` have `bytes` of dynamic shared memory on the current device.  (Threads that come here
    // together set the same value; what failed is tried again by the next call.)
    cudaError_t operator()(const void* kern, int bytes)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;      // (others: set by every call)
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }

private:
    std::atomic<uint64_t> done_{0};      // devices that are done
};

}  // namespace pa

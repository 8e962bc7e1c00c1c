// Host code that runs once on each device: a kernel's attributes belong to the device that is current when they are set.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace ds {

class OncePerDevice {
    static constexpr int kDevices = 64;  // devices past these: on every call
    std::atomic<bool> done_[kDevices] = {};

  public:
    // f() unless it has succeeded on the current device.
    template <typename F>
    cudaError_t operator()(F f) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool kept = dev >= 0 && dev < kDevices;
        if (kept && done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
        e = f();
        if (kept && e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
        return e;
    }
};

}  // namespace ds

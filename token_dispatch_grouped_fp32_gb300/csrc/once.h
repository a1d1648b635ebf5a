// once.h -- what a launcher sets up on a device before its first launch there.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace moe {

// setup(device), until it has succeeded once on the current device.  Host
// threads whose first calls meet may each run it: it writes the same values
// whoever comes first, to atomics, and a thread that skips it has seen all that
// a finished one wrote.  (No lock: nothing that can throw at a C entry, and a
// setup that failed is tried again by the next call.)
class OncePerDevice {
  public:
    static constexpr int kDevices = 64;
    template <typename F> cudaError_t operator()(F setup) {
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
        if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
        if ((err = setup(dev)) != cudaSuccess) return err;
        done_[dev].store(true, std::memory_order_release);
        return cudaSuccess;
    }

  private:
    std::atomic<bool> done_[kDevices] = {};
};

}  // namespace moe

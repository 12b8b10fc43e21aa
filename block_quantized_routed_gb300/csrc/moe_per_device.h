// What the host keeps per device: attributes and settings of a kernel hold for
// the device that was current when they were asked for or made.
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace moe {

// A number per device, 0 where it is not known yet.  Host threads may call at
// the same time: then `get` may be asked more than once.
class PerDevice {
 public:
  // The current device's number: kept, or what get(device) gives (kept unless it is 0).
  template <typename F>
  int operator()(F get) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    if (dev < 0 || dev >= kDevices) return get(dev);
    int v = v_[dev].load(std::memory_order_acquire);
    if (v == 0) {
      v = get(dev);
      v_[dev].store(v, std::memory_order_release);
    }
    return v;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> v_[kDevices] = {};
};

}  // namespace moe

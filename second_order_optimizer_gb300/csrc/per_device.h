// Host state that CUDA keeps per device.
#pragma once
#include <atomic>

namespace kfac {

// Runs set() the first time on each device, and again while it fails there: a kernel's
// attributes belong to the device that is current when they are set.
class OncePerDevice {
  static constexpr int kMax = 64;
  std::atomic<bool> done_[kMax] = {};

 public:
  template <typename Set> bool operator()(int dev, Set set) {
    if (dev < 0 || dev >= kMax) return set();
    if (done_[dev].load(std::memory_order_acquire)) return true;
    if (!set()) return false;
    done_[dev].store(true, std::memory_order_release);
    return true;
  }
};

}  // namespace kfac

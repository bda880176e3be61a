// A set-up step that each device needs once, such as a kernel's shared-memory
// limit.  Only success is remembered: a step that failed is taken again.
#pragma once

#include <atomic>
#include <cstdint>

namespace wq {

class OncePerDevice {
  std::atomic<uint64_t> done_{0};  // a bit per device

 public:
  // devices 0 .. 63; `set` may run twice where threads meet in it
  template <class Set>
  bool operator()(int device, Set &&set) {
    const uint64_t bit = uint64_t(1) << device;
    if (done_.load(std::memory_order_relaxed) & bit) return true;
    if (!set()) return false;
    done_.fetch_or(bit, std::memory_order_relaxed);
    return true;
  }
};

}  // namespace wq

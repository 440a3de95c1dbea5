// What a launcher learns from the runtime once per device and keeps.
#pragma once

#include <atomic>

namespace moe {

// A positive number per device.  Threads that call at the same time each learn
// it, and publish the same value; a thread sees a whole value or none.
class PerDevice {
 public:
  // The device's number: what learn() returned the first time, if it was positive.
  template <class F>
  int get(int dev, F learn) {
    if (dev < 0 || dev >= MAX) return learn();
    int v = v_[dev].load(std::memory_order_acquire);
    if (v > 0) return v;
    v = learn();
    if (v > 0) v_[dev].store(v, std::memory_order_release);
    return v;
  }

 private:
  static constexpr int MAX = 64;
  std::atomic<int> v_[MAX] = {};
};

}  // namespace moe

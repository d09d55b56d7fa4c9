// per_device.h -- values that are found out once per device (occupancy, attributes), by
// whichever thread needs them first.  Host code without CUDA types.
#pragma once
#include <atomic>
#include <mutex>

namespace fgf8 {

constexpr int kMaxDevices = 64;

// get() publishes a value only when it is complete: the flag is released after the fill and
// acquired before the value is read, so a thread that makes its first call beside another
// one's never sees half of it.  A fill that fails is tried again by the next call.
template <typename T>
class PerDevice {
 public:
  // fill(T&) returns 0 or an error code, which get() passes on.  dev is below kMaxDevices.
  template <typename Fill>
  int get(int dev, const T** out, Fill&& fill) {
    Slot& s = slots_[dev];
    if (!s.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mutex_);
      if (!s.ready.load(std::memory_order_relaxed)) {
        if (const int r = fill(s.value)) return r;
        s.ready.store(true, std::memory_order_release);
      }
    }
    *out = &s.value;
    return 0;
  }

 private:
  struct Slot {
    std::atomic<bool> ready{false};
    T value{};
  };
  Slot slots_[kMaxDevices];
  std::mutex mutex_;
};

}  // namespace fgf8

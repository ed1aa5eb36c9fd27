// q4k_device_once.h — what a process does once for each device (a kernel's shared memory attribute),
// asked for before every launch from any thread.
#pragma once
#include <atomic>

namespace q4k {

class DeviceOnce {
 public:
  // f() on the current device `dev`, unless an earlier f() for it returned `ok`; returns its result.  Threads
  // that come at the same time may each run f(), which has to be harmless when it runs again.
  template <class F, class R>
  R run(int dev, R ok, F&& f) {
    const bool known = dev >= 0 && dev < kDevices;
    if (known && done_[dev].load(std::memory_order_acquire)) return ok;
    const R r = f();
    if (known && r == ok) done_[dev].store(true, std::memory_order_release);
    return r;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> done_[kDevices] = {};
};

}  // namespace q4k

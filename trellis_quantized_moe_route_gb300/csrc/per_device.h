// What a process sets once for each device.
#pragma once

#include <stdint.h>

#include <atomic>

namespace tmoe {

// Calls f() the first time for each device and until it succeeds; returns its
// error (0: done, now or before). Threads that come at once may both call it. A
// device past the 64 that have a bit gets the call every time.
class OncePerDevice {
 public:
  template <typename F>
  auto operator()(int device, F f) -> decltype(f()) {
    const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
    if (done_.load(std::memory_order_acquire) & bit) return decltype(f())(0);
    const auto e = f();
    if (e == decltype(f())(0)) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace tmoe

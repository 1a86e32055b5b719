// What a process does once per device: a kernel's attributes belong to the device that is current when they
// are set, so a second device needs them again. Host only, no CUDA.
#pragma once

#include <atomic>
#include <cstdint>

namespace mxq {

class PerDevice {
 public:
  // Runs `f` (0: it succeeded) for a device for which it has not succeeded yet; its result, or 0. Two
  // threads may both run it. Devices past the 64th run it every time.
  template <typename F>
  auto once(int device, F&& f) -> decltype(f()) {
    const uint64_t bit = device >= 0 && device < 64 ? uint64_t(1) << device : 0;
    if ((done_.load(std::memory_order_acquire) & bit) != 0) return {};
    const auto r = f();
    if (r == decltype(f()){}) done_.fetch_or(bit, std::memory_order_release);
    return r;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

}  // namespace mxq

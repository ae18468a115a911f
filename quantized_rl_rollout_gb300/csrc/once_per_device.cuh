// A setting that each device of the process needs once, such as a kernel's limit of
// dynamic shared memory.
#pragma once

#include <stdint.h>

#include <atomic>

namespace qrr {

class OncePerDevice {
  std::atomic<uint64_t> done_{0};  // a bit a device; devices from 64 on are set each time

 public:
  // set(), unless it has succeeded (returned 0) on device `dev`.
  template <class F>
  auto operator()(int dev, F set) -> decltype(set()) {
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (done_.load(std::memory_order_acquire) & bit) return static_cast<decltype(set())>(0);
    const auto e = set();
    if (e == 0) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

}  // namespace qrr

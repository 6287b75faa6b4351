// Set-up that belongs to a device, such as a kernel's opt-in to large dynamic
// shared memory: done at the first call on each device and not again.
#pragma once

#include <atomic>
#include <cstdint>

namespace sgl {

class PerDevice {
  public:
    // 0 when device `dev` is set up: set() (0, or an error code) has succeeded
    // for it, now or before.  An error is returned and tried again by the next
    // call.  Threads that meet here for the first time may each call set().
    template <class Set>
    int ready(int dev, Set set) {
        const bool kept = dev >= 0 && dev < 64;
        const uint64_t bit = kept ? uint64_t(1) << dev : 0;
        if (done_.load(std::memory_order_acquire) & bit) return 0;
        const int e = set();
        if (!e && kept) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }

  private:
    std::atomic<uint64_t> done_{0};
};

}  // namespace sgl

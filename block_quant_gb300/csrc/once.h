// Set-up that a device needs once per process, such as kernel attributes, which belong to
// the device they were set on.
#pragma once

#include <atomic>
#include <mutex>

namespace bq {

// run(dev, set_up): every caller returns after the device's set-up is done, whichever
// thread did it.  set_up returns 0 or an error code, which its caller gets; one that failed
// is tried again by the next call.  A device outside [0, 64) is set up by every call.
class OncePerDevice {
 public:
  template <typename F>
  int run(int dev, F set_up) {
    if (dev < 0 || dev >= kDevices) return set_up();
    if (done_[dev].load(std::memory_order_acquire)) return 0;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev].load(std::memory_order_relaxed)) return 0;
    const int rc = set_up();
    if (rc == 0) done_[dev].store(true, std::memory_order_release);
    return rc;
  }

 private:
  static constexpr int kDevices = 64;
  std::mutex mu_;
  std::atomic<bool> done_[kDevices] = {};
};

}  // namespace bq

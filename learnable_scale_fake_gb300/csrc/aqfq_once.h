// aqfq_once.h -- a kernel's attributes (its shared-memory limit, its cluster size) belong to
// the device that is current when they are set: they are set once per device, at the kernel's
// first launch there.  Host only, no CUDA header.
#pragma once

#include <atomic>

namespace aqfq {

class DeviceOnce {
 public:
  static constexpr int kMost = 256;
  // set() returns 0 on success; run returns what it returned.  It is called by the first run
  // for a device and again after a failure, and by every run for an ordinal out of range.
  // Two threads may both call it: setting an attribute twice is the same as once.
  template <typename F>
  int run(int dev, F set) {
    if (dev < 0 || dev >= kMost) return int(set());
    if (done_[dev].load(std::memory_order_acquire)) return 0;
    const int e = int(set());
    if (e == 0) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<bool> done_[kMost] = {};
};

}  // namespace aqfq

// What the host keeps for each device between launches: SM counts, occupancies
// and whether a kernel's attributes are set, all of which are a device's own.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace moe4 {

constexpr int kMaxDevices = 64;  // devices are numbered below it

static inline int current_device() {
  int dev = 0;
  return (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices) ? dev : 0;
}

// A positive number for each device, found by `find` when it is first needed
// there. Threads that come first together all find it, and the same; what
// `find` has set up is visible to whoever reads the number. One that is not
// positive is a failure, which is not kept.
class PerDevice {
  std::atomic<int> n_[kMaxDevices] = {};

 public:
  template <typename F>
  int get(F find) {
    std::atomic<int> &kept = n_[current_device()];
    int n = kept.load(std::memory_order_acquire);
    if (n <= 0) {
      n = find();
      if (n > 0) kept.store(n, std::memory_order_release);
    }
    return n;
  }
};

// SM count of the current device.
static inline int sm_count() {
  static PerDevice sms;
  return sms.get([] {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, current_device()) != cudaSuccess || n <= 0) n = 148;
    return n;
  });
}

}  // namespace moe4

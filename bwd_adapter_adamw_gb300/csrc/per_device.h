// What the runtime keeps for each device (a kernel's attributes, how many of its clusters are resident
// at once) is remembered for each device: a process may use several. No CUDA here, so that a host
// test can compile it.
#pragma once

#include <atomic>
#include <cstdint>

namespace lora {

constexpr int kDevices = 64;   // remembered; a device past them is asked for every time

// f() once per device, until it has succeeded there (returned `good`). Two threads may both run it.
template <typename E, typename F>
E once_on_device(std::atomic<uint64_t>& done, int dev, E good, F f) {
  if (dev < 0 || dev >= kDevices) return f();
  const uint64_t bit = uint64_t(1) << dev;
  if (done.load(std::memory_order_acquire) & bit) return good;
  const E e = f();
  if (e == good) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// N values per device, each found by f() (not negative; negative: not known, found again next time).
template <int N>
struct DeviceValues {
  std::atomic<int> v[kDevices][N] = {};   // value + 1; 0: not known
  template <typename F>
  int get(int dev, int i, F f) {
    if (dev < 0 || dev >= kDevices) return f();
    int n = v[dev][i].load(std::memory_order_relaxed);
    if (n == 0) {
      n = f() + 1;
      if (n > 0) v[dev][i].store(n, std::memory_order_relaxed);
    }
    return n - 1;
  }
};

}  // namespace lora

// A positive number asked once for each device, from any host thread.
#pragma once
#include <atomic>

struct PerDevice {
  static constexpr int N = 64;   // devices from the 65th on are asked about every time
  std::atomic<int> v[N];         // 0: not known yet
};

// ask(dev) gives the number, or 0 where that failed (asked again next time).  Two
// threads that come first at once both ask, and store the same.
template <class Ask>
int per_device(PerDevice& c, int dev, Ask ask) {
  if (dev < 0 || dev >= PerDevice::N) return ask(dev);
  int x = c.v[dev].load(std::memory_order_acquire);
  if (x == 0) {
    x = ask(dev);
    if (x > 0) c.v[dev].store(x, std::memory_order_release);
  }
  return x;
}

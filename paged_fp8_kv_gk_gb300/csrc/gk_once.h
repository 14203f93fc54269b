// gk_once.h -- what the library sets up once a device (kernel attributes, grid
// sizes), by the first call that needs it, from any host thread.
#pragma once

#include <atomic>
#include <mutex>

namespace gk {

template <typename T, int kDevices>
class PerDevice {
 public:
  static constexpr int devices = kDevices;
  // setup(T&) -> E, E{} being success: run once for device `dev`; the threads
  // that come meanwhile wait for it, later ones only read `ready`, whose release
  // and acquire make every field visible with it.  A setup that failed has left
  // nothing behind and is tried again by the next call.
  template <typename E, typename F>
  E get(int dev, const T** out, F setup) {
    Slot& s = slots_[dev];
    if (!s.ready.load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> hold(s.lock);
      if (!s.ready.load(std::memory_order_relaxed)) {
        T value{};
        const E e = setup(value);
        if (e != E{}) return e;
        s.value = value;
        s.ready.store(true, std::memory_order_release);
      }
    }
    *out = &s.value;
    return E{};
  }

 private:
  struct Slot {
    std::mutex lock;
    std::atomic<bool> ready{false};
    T value{};
  };
  Slot slots_[kDevices];
};

}  // namespace gk

// What a launch finds out or sets once a device: a kernel's attributes belong to
// the device's context, and its occupancy to the device.
#pragma once
#include <mutex>

namespace moe {

template <typename T>
class PerDevice {
 public:
  // make()'s result for device `dev`, made by the first call that asks (each time past
  // the devices that are kept).  Safe from several host threads.
  template <typename F>
  T get(int dev, F make) {
    if (dev < 0 || dev >= kDevices) return make();
    Slot &s = slots_[dev];
    std::call_once(s.once, [&] { s.value = make(); });
    return s.value;
  }

 private:
  static constexpr int kDevices = 64;
  struct Slot {
    std::once_flag once;
    T value;
  };
  Slot slots_[kDevices];
};

}  // namespace moe

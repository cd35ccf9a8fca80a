// What has to be set up once on every device that a kernel is launched on: function attributes belong to a
// device, and so do the counts of resident blocks.
#pragma once

#include <mutex>

namespace poetx {

template <typename T>
class PerDevice {
 public:
  static constexpr int kDevices = 64;
  // set_up()'s answer on this device: made on the first call, kept for the later ones (a device without a place
  // here: made every time).
  template <typename F>
  T get(int device, F set_up) {
    if (device < 0 || device >= kDevices) return set_up();
    Entry& e = entries_[device];
    std::call_once(e.once, [&] { e.value = set_up(); });
    return e.value;
  }

 private:
  struct Entry {
    std::once_flag once;
    T value{};
  };
  Entry entries_[kDevices];
};

}  // namespace poetx

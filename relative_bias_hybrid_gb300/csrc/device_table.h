// device_table.h -- small positive numbers that were asked of the runtime once for each device
// (clusters that are resident at once, say): a value belongs to the device that was current
// when it was asked for.
//
// Plain C++ without CUDA types, so that its logic can be checked on a machine without a GPU.
#pragma once

#include <atomic>

namespace inkattn {

template <int kDevices, int kSlots>
class DeviceTable {
  public:
    // The number of `device` and `slot`; lookup() is called until it has given a positive one.  A
    // device beyond the table is asked every time.
    template <class Lookup>
    int get(int device, int slot, Lookup &&lookup) {
        if (device < 0 || device >= kDevices || slot < 0 || slot >= kSlots) return lookup();
        std::atomic<int> &known = vals_[device][slot];
        int n = known.load(std::memory_order_relaxed);
        if (n > 0) return n;
        n = lookup();
        if (n > 0) known.store(n, std::memory_order_relaxed);
        return n;
    }

  private:
    std::atomic<int> vals_[kDevices][kSlots] = {};
};

}  // namespace inkattn

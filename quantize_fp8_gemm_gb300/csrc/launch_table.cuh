// launch_table.cuh -- what launches keep of a kernel from call to call.  Host code only.
#pragma once

#include <atomic>

namespace fp8q {

constexpr int kMaxDevices = 64;  // devices of a process that tables are kept for

// A positive number for each device and launch size (below SIZES), asked for once.
// Both parts of an answer belong to one device: how many CTAs of a kernel run at a
// time, and the attributes that were set on that device's copy of it on the way.
template <int SIZES>
class DeviceTable {
  public:
    // *value = the number of (device, size); ask(value) gives it the first time and
    // returns an error code, 0 for success.  An error is not kept.
    template <typename Ask>
    auto get(int device, int size, int* value, Ask&& ask) -> decltype(ask(value)) {
        using Error = decltype(ask(value));
        const bool kept = device >= 0 && device < kMaxDevices;
        if (kept && (*value = known_[device][size].load(std::memory_order_acquire)) > 0) return Error(0);
        const Error e = ask(value);
        if (kept && e == Error(0)) known_[device][size].store(*value, std::memory_order_release);
        return e;
    }

  private:
    std::atomic<int> known_[kMaxDevices][SIZES] = {};
};

}  // namespace fp8q

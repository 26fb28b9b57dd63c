// kda_per_device.h -- what is found out once for each device (host side).
#pragma once

#include <atomic>

namespace kda {

// A number above 0 that depends on a device and a kernel alone: how many blocks
// run at once, or that an attribute was set.  Threads that come first together
// all find it, and the same; errors and 0 are not kept.
class PerDevice {
public:
    // find(int&) gives the number or an error (other than 0); `out` is the number of `device`.
    template <typename F>
    auto get(int device, int& out, F find) -> decltype(find(out)) {
        const bool kept = device >= 0 && device < kDevices;
        out = kept ? value_[device].load(std::memory_order_acquire) : 0;
        if (out > 0) return decltype(find(out))(0);
        int found = 0;
        const auto e = find(found);
        out = found;
        if (kept && e == decltype(find(out))(0)) value_[device].store(found, std::memory_order_release);
        return e;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> value_[kDevices] = {};
};

}  // namespace kda

// What a call finds out once per device (attributes set, occupancy), shared by
// the host threads that call the library.  Plain C++.
#pragma once
#include <atomic>
#include <mutex>

namespace razer {

// The first get() of a device runs `fill`, which returns whether it could tell;
// every other one, of any thread, sees the whole value it left.  A failed fill
// is tried again by the next call.  (Plain stores are not enough: a thread that
// saw half of a table chose another split of K, and so another order of sums.)
template <typename T> class PerDevice {
    static constexpr int kDevices = 64;
    std::atomic<bool> known[kDevices] = {};
    T values[kDevices] = {};
    std::mutex filling;

public:
    template <typename Fill> bool get(int dev, T &out, Fill fill)
    {
        if (dev < 0 || dev >= kDevices) return fill(out);
        if (!known[dev].load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> hold(filling);
            if (!known[dev].load(std::memory_order_relaxed)) {
                T v = {};
                if (!fill(v)) return false;
                values[dev] = v;
                known[dev].store(true, std::memory_order_release);
            }
        }
        out = values[dev];
        return true;
    }
};

}  // namespace razer

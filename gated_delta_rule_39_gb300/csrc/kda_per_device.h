// What has to be set once on every device (a kernel's attributes): plain C++, no CUDA call.
#pragma once
#include <atomic>

namespace kda {

constexpr int kMaxDeviceIndex = 64;

class OncePerDevice {
public:
    // Calls set() unless it has succeeded for this device before; returns 0, or what set()
    // returned when it failed (the next call then tries again).  Threads that come at the same
    // time may both call it.
    template <class F>
    auto operator()(int device, F&& set) -> decltype(set()) {
        using Result = decltype(set());
        if (done_[device].load(std::memory_order_acquire)) return Result(0);
        const Result r = set();
        if (r == Result(0)) done_[device].store(true, std::memory_order_release);
        return r;
    }

private:
    std::atomic<bool> done_[kMaxDeviceIndex] = {};
};

}  // namespace kda

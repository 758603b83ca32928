// device_setup.h -- what a launch sets up once a device (a kernel's attributes, what
// the device holds of it).  Plain C++.
#pragma once

#include <atomic>
#include <mutex>

namespace fp8w {

// The set-up of one kernel on each device: done by the first call, and where it failed
// by the next one again, which returns its error then, so that nothing is launched
// without it.
class DeviceSetup {
public:
    // f returns an error code, 0 for success.
    template <class F>
    auto operator()(int device, F&& f) -> decltype(f()) {
        using Error = decltype(f());
        if (device < 0 || device >= kDevices) return f();
        if (done_[device].load(std::memory_order_acquire)) return Error{};
        std::lock_guard<std::mutex> lock(busy_);
        if (done_[device].load(std::memory_order_relaxed)) return Error{};
        const Error e = f();
        if (e == Error{}) done_[device].store(true, std::memory_order_release);
        return e;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<bool> done_[kDevices] = {};
    std::mutex busy_;
};

}  // namespace fp8w

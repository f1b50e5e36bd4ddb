// per_device.h -- host state that belongs to a device, not to the process.
#pragma once

#include <atomic>

namespace nm {

constexpr int kMaxDevices = 64;

// Does something for each device until it has succeeded there once. Threads may do it at the same
// time (what is done is the same each time); a failure is not kept.
class OncePerDevice {
public:
    template <class F> bool operator()(int device, const F &f)
    {
        if (device < 0 || device >= kMaxDevices)
            return false;
        if (done_[device].load(std::memory_order_acquire))
            return true;
        if (!f())
            return false;
        done_[device].store(true, std::memory_order_release);
        return true;
    }

private:
    std::atomic<bool> done_[kMaxDevices] = {};
};

} // namespace nm

// What has to be set once per device.  Host code without HIP, so that it can be
// tested without a device.
#pragma once

#include <atomic>

namespace fa {

class DeviceOnce {
public:
    // Runs `set` unless it has succeeded for this device.  Returns its status,
    // 0 for success: a failure is reported and tried again by the next call.
    // Threads that race set the same value twice; devices beyond the table set
    // it on every call.
    template <typename F> int run(int device, F set)
    {
        const bool known = device >= 0 && device < DEVICES;
        if (known && done_[device].load(std::memory_order_acquire))
            return 0;
        const int status = set();
        if (known && status == 0)
            done_[device].store(true, std::memory_order_release);
        return status;
    }

private:
    static constexpr int DEVICES = 64;
    std::atomic<bool> done_[DEVICES] = {};
};

} // namespace fa

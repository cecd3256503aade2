// What a kernel needs once on each device before its first launch there
// (function attributes, the number of SMs).  No CUDA in here.
#pragma once

#include <atomic>
#include <mutex>

namespace bsa {

constexpr int kMaxDevices = 64;

// Host threads may make their first calls at the same time: one of them runs the
// set-up, the others wait for it, and whoever is told that it is done sees what it
// wrote.  A set-up that fails is tried again by the next call.
class DeviceSetup {
public:
    // True once setup() has returned true for the device.
    template <typename Setup>
    bool once(int dev, Setup&& setup) {
        if (dev < 0 || dev >= kMaxDevices) return false;
        if (done_[dev].load(std::memory_order_acquire)) return true;
        std::lock_guard<std::mutex> hold(lock_);
        if (done_[dev].load(std::memory_order_relaxed)) return true;
        if (!setup()) return false;
        done_[dev].store(true, std::memory_order_release);
        return true;
    }

private:
    std::mutex lock_;
    std::atomic<bool> done_[kMaxDevices] = {};
};

}  // namespace bsa

// What has to be found out or set once for every device that a process uses.
#pragma once

#include <atomic>
#include <mutex>

namespace clef {

// One value a device.  get() has `make(&value)` fill it at the device's first call; make returns 0, or an
// error, which get() passes on without keeping it: the next call tries again.  Several threads may call.
template <typename T>
class PerDevice {
public:
    template <typename Make>
    int get(int device, T* out, Make make) {
        if (device < 0 || device >= kMost) return make(out);  // not kept
        if (!ready_[device].load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> lock(mutex_);
            if (!ready_[device].load(std::memory_order_relaxed)) {
                const int error = make(&value_[device]);
                if (error) return error;
                ready_[device].store(true, std::memory_order_release);
            }
        }
        *out = value_[device];
        return 0;
    }

private:
    static constexpr int kMost = 64;
    std::mutex mutex_;
    std::atomic<bool> ready_[kMost] = {};
    T value_[kMost] = {};
};

}  // namespace clef

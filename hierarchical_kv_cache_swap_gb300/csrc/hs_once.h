// A value for each device, made once (host code).
#pragma once

#include <atomic>
#include <mutex>

namespace hs {

template <class T>
class PerDevice {
public:
    static constexpr int kDevices = 64;

    // The device's value (0 <= device < kDevices). The first call makes it with make(T*), which
    // returns 0, or an error that this call returns and the next one tries again after. Calls
    // from other threads meanwhile wait; later ones take no lock.
    template <class F>
    int get(int device, F make, const T** value) {
        if (!ready_[device].load(std::memory_order_acquire)) {
            std::lock_guard<std::mutex> hold(lock_);
            if (!ready_[device].load(std::memory_order_relaxed)) {  // another thread made it meanwhile
                if (const int error = make(&values_[device])) return error;
                ready_[device].store(true, std::memory_order_release);
            }
        }
        *value = &values_[device];
        return 0;
    }

private:
    std::mutex lock_;
    std::atomic<bool> ready_[kDevices] = {};
    T values_[kDevices];
};

}  // namespace hs

// A limit per device that launches raise as they need it: the dynamic shared
// memory that a kernel may ask for.
#pragma once

#include <atomic>
#include <mutex>

namespace pkv {

// Launches of one kernel with different sizes may come from several threads.
// The limit is only ever raised, and what is known of it changes together with
// it: a launch whose size was found to be within the limit stays within it.
class RaisedLimit {
public:
    static constexpr int kDevices = 64;  // the library refuses further ones

    // Makes the limit of `device` at least `value` by set(value), which returns 0
    // or an error; calls nothing if it is that high already (so that launches
    // captured in a CUDA graph, after one that was not, make no attribute calls).
    template <class Set>
    auto at_least(int device, int value, Set set) -> decltype(set(value)) {
        if (known_[device].load(std::memory_order_acquire) >= value) return {};
        std::lock_guard<std::mutex> lock(mutex_);
        if (known_[device].load(std::memory_order_relaxed) >= value) return {};
        const auto e = set(value);
        if (e == decltype(set(value)){}) known_[device].store(value, std::memory_order_release);
        return e;
    }

private:
    std::mutex mutex_;
    std::atomic<int> known_[kDevices] = {};
};

}  // namespace pkv

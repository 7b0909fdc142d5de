// What has to be set once on every device, as a kernel's shared-memory limit has (the
// attribute belongs to the kernel as loaded on one device).
#pragma once

#include <atomic>

namespace zha {

class OncePerDevice {
    std::atomic<unsigned long long> done_{0};  // bit i: set on device i

public:
    // Runs set() unless it has succeeded for `device` before; returns its result (0: success).
    // From several threads at once it may run more than once.
    template <typename F>
    auto operator()(int device, F set) -> decltype(set()) {
        using Result = decltype(set());
        const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0;
        if (done_.load(std::memory_order_acquire) & bit) return Result(0);
        const Result r = set();
        if (r == Result(0)) done_.fetch_or(bit, std::memory_order_release);
        return r;
    }
};

}  // namespace zha

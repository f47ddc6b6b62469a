// Work that is needed once on every device of a process, such as the attributes of a kernel, which
// belong to the device that was current when they were set.
#pragma once

#include <atomic>
#include <cstdint>

namespace idx {

class PerDevice {
    std::atomic<uint64_t> done_{0};

public:
    // f() on `device`, which is current, unless it has returned 0 there before; its result.
    template <typename F> int run(int device, F&& f) {
        const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
        if (done_.load(std::memory_order_acquire) & bit) return 0;
        const int e = f();
        if (e == 0) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

}  // namespace idx

// A fact about a device that costs a query (how many clusters of a kernel run at once, where
// shared memory starts), asked for once per device. Host code without CUDA headers.
#pragma once

#include <atomic>

namespace qnf4 {

class DeviceCache {
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices] = {};                  // 0: not asked yet

  public:
    // The fact for device number dev: ask() the first time. Facts are positive; what ask() returns
    // otherwise (a failed query) is passed on and not kept, and devices past the array are asked each
    // time. Threads that ask at once get the same fact.
    template <typename Ask>
    int get(int dev, Ask ask) {
        const bool kept = dev >= 0 && dev < kDevices;
        int v = kept ? known_[dev].load(std::memory_order_relaxed) : 0;
        if (v == 0) {
            v = ask();
            if (kept && v > 0) known_[dev].store(v, std::memory_order_relaxed);
        }
        return v;
    }
};

}  // namespace qnf4

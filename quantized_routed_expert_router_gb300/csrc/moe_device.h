// moe_device.h - answers that hold for a device as long as the process lives.
#pragma once

#include <atomic>

namespace moe {

// ask() is called until it has an answer, a number that is not negative; -1: none this time, and the next call asks again.
// One object a question; host threads may ask at once.
class PerDevice {
public:
    template <typename F>
    int get(int device, F ask) {
        if (device < 0 || device >= kDevices) return ask();
        int n = known_[device].load(std::memory_order_relaxed) - 1;
        if (n < 0) {
            n = ask();
            if (n >= 0) known_[device].store(n + 1, std::memory_order_relaxed);
        }
        return n;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices] = {};   // the answer and 1; 0: not known
};

}  // namespace moe

// asked.cuh -- a number asked of the driver once, in plain C++.
#pragma once

#include <atomic>

namespace kvc {

// Asks until it is told: an answer of 0 or less is a failure (memory that ran out
// while the driver brought the code in, say), which the next call may not meet, so
// it is not kept.
class AskedOnce {
public:
    template <typename F>
    int get(F ask) {
        int n = told_.load(std::memory_order_relaxed);
        if (n <= 0) {
            n = ask();
            if (n > 0) told_.store(n, std::memory_order_relaxed);
        }
        return n;
    }

private:
    std::atomic<int> told_{0};
};

}  // namespace kvc

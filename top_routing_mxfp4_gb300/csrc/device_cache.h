// Answers about a device, each asked once: positive numbers by device and
// question.  A question that fails (an answer of 0 or less) is not remembered;
// neither is one about a device beyond the table.  Host code, any thread.
#pragma once

#include <atomic>

namespace lmoe {

template <int QUESTIONS>
class DeviceCache {
public:
    static constexpr int DEVICES = 32;
    // The answer, or 0; question in [0, QUESTIONS).
    template <typename Ask>
    int get(int device, int question, Ask ask)
    {
        std::atomic<int> *at = device >= 0 && device < DEVICES ? &known[device][question] : nullptr;
        int n = at ? at->load(std::memory_order_relaxed) : 0;
        if (n > 0) return n;
        n = ask();
        if (n <= 0) return 0;
        if (at) at->store(n, std::memory_order_relaxed);
        return n;
    }

private:
    std::atomic<int> known[DEVICES][QUESTIONS] = {};
};

}  // namespace lmoe

// Answers of a device to questions that it always answers alike, each asked once.
#pragma once

#include <atomic>

constexpr int kSsdMaxDevices = 64;

// The answers to kKeys questions of every device (statically zero: none asked yet).
template <int kKeys>
struct SsdAnswers {
    std::atomic<int> known[kSsdMaxDevices][kKeys];      // the answer plus one; 0: not asked yet

    // Answer number `key` of `device`: a known one, or ask()'s, which is kept unless it is
    // negative (a failure, to be asked again by the next call).
    template <typename Ask>
    int get(int device, int key, Ask &&ask) {
        const bool keep = device >= 0 && device < kSsdMaxDevices;
        if (keep) {
            const int n = known[device][key].load(std::memory_order_relaxed);
            if (n > 0) return n - 1;
        }
        const int n = ask();
        if (keep && n >= 0) known[device][key].store(n + 1, std::memory_order_relaxed);
        return n;
    }
};

// Threads in place of CTAs: each writes the statuses it owns, then leaves through settle.h. Arguments: rounds, seed.
// Exits 0 if after every round the sequences of the CTAs that gave up, and only those, are marked, and every word is zero.
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <thread>
#include <vector>

#include "settle.h"

constexpr int kCtas = 12, kSeqs = 40, kTimeout = 6;

struct Memory {
    std::atomic<int> words[2 * kCtas] = {}, any{0}, done{0}, status[kSeqs] = {};
    void put(int i, int v) { words[i].store(v, std::memory_order_relaxed); }
    int get(int i) { return words[i].load(std::memory_order_relaxed); }
    void raise() { any.store(1, std::memory_order_relaxed); }
    bool raised() { return any.load(std::memory_order_relaxed); }
    void lower() { any.store(0, std::memory_order_relaxed); }
    void fence() { std::atomic_thread_fence(std::memory_order_seq_cst); }
    int count() { return done.fetch_add(1, std::memory_order_relaxed); }
    void clear_count() { done.store(0, std::memory_order_relaxed); }
    void mark(int b) { status[b].store(kTimeout, std::memory_order_relaxed); }
};

int main(int argc, char** argv) {
    std::mt19937 rng(argc > 2 ? std::atoi(argv[2]) : 1);
    static Memory m;
    for (int round = 0, n = argc > 1 ? std::atoi(argv[1]) : 100; round < n; ++round) {
        bool late[kCtas];
        int pause[kCtas], begin[kCtas + 1] = {};
        for (int i = 0; i < kCtas; ++i) {
            late[i] = rng() % 4 == 0 && round % 3;
            pause[i] = rng() % 200;
            begin[i + 1] = i + 1 == kCtas ? kSeqs : begin[i] + (int)(rng() % 7) * (begin[i] + 6 < kSeqs);
        }
        for (auto& s : m.status) s = -7;
        std::vector<std::thread> t;
        for (int i = 0; i < kCtas; ++i)
            t.emplace_back([&, i] {
                for (volatile int k = 0; k < pause[i] * 50; k = k + 1) {
                }
                for (int b = i; b < kSeqs; b += kCtas) m.status[b].store(b % 3 ? 0 : 4, std::memory_order_relaxed);
                // a run shares its first sequence with the run before
                const int b0 = begin[i] ? begin[i] - 1 : 0, b1 = begin[i + 1];
                specv::settle(m, i, kCtas, late[i] ? b0 : 0, late[i] ? b1 : 0);
            });
        for (auto& x : t) x.join();
        for (int b = 0; b < kSeqs; ++b) {
            bool marked = false;
            for (int i = 0; i < kCtas; ++i) marked |= late[i] && b >= (begin[i] ? begin[i] - 1 : 0) && b < begin[i + 1];
            if (m.status[b] != (marked ? kTimeout : b % 3 ? 0 : 4)) return std::printf("round %d sequence %d: %d\n", round, b, (int)m.status[b]), 1;
        }
        for (auto& w : m.words)
            if (w) return std::printf("round %d: a word is left\n", round), 1;
        if (m.any || m.done) return std::printf("round %d: a count is left\n", round), 1;
    }
    return 0;
}

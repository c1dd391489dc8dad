// The meetings of the tensor-memory attention kernel's softmax warps (kvl_attend_meet.cuh) with a thread for
// each warp and named barriers that count arrivals as the hardware does.  A thread's bounded waits run out at
// random; whatever the moment, every thread has to come to the end and every barrier to be empty then.
#include <atomic>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#define __host__
#define __device__
#define __forceinline__ inline
#include "kvl_attend_meet.cuh"

namespace {

struct Barriers {
    std::mutex m;
    std::condition_variable cv;
    int count[16] = {}, phase[16] = {};

    bool add(int id, int n)  // whether the barrier is complete
    {
        count[id] += 32;
        if (count[id] < n) return false;
        if (count[id] > n) {
            std::printf("barrier %d: %d arrivals of %d\n", id, count[id], n);
            std::fflush(stdout);
            std::_Exit(1);
        }
        count[id] = 0;
        ++phase[id];
        cv.notify_all();
        return true;
    }
    void arrive(int id, int n)
    {
        std::lock_guard<std::mutex> l(m);
        add(id, n);
    }
    void wait(int id, int n)
    {
        std::unique_lock<std::mutex> l(m);
        const int before = phase[id];
        if (add(id, n)) return;
        if (!cv.wait_for(l, std::chrono::seconds(10), [&] { return phase[id] != before; })) {
            std::printf("barrier %d: left waiting with %d arrivals of %d\n", id, count[id], n);
            std::fflush(stdout);
            std::_Exit(1);
        }
    }
};

struct Meet {
    Barriers *b;
    template <int N> void wait(int id) const { b->wait(id, N); }
    template <int N> void arrive(int id) const { b->arrive(id, N); }
};

struct Trial {
    Barriers bars;
    std::atomic<int> gone{0};
    // what the kernel's memory barriers carry: steps whose K, V are converted, whose scores are there, whose products
    // are issued, by tile
    std::atomic<int> k_full{0}, v_full{0}, scores[2] = {{0}, {0}}, values[2] = {{0}, {0}};
    int n, chance;
    unsigned first;  // steps of earlier jobs
    bool two;

    struct Warp {
        Trial &t;
        std::mt19937 rng;
        // a bounded wait: true once `ready` holds, false when another has given up or the wait runs out
        template <typename F>
        bool wait(F ready)
        {
            for (int tries = 1;; ++tries) {
                if (ready()) return true;
                if (tries % 4 == 0) {
                    if (t.gone) return false;
                    if (int(rng() % 20000) < t.chance) {
                        t.gone = 1;
                        return false;
                    }
                }
                std::this_thread::yield();
            }
        }
        void pause()
        {
            for (int k = rng() % 4; k; --k) std::this_thread::yield();
        }
    };

    void convert(unsigned seed)
    {
        Warp w{*this, std::mt19937(seed)};
        auto used = [&](std::atomic<int> (&x)[2], int s) { return x[0] > s && (!two || x[1] > s); };
        for (int s = 0; s < n; ++s) {
            if (!w.wait([&] { return s < 2 || used(scores, s - 2); })) break;
            k_full = s + 1;
            w.pause();
            if (!w.wait([&] { return s < 2 || used(values, s - 2); })) break;
            v_full = s + 1;
        }
    }

    void softmax(int g, int warp, unsigned seed)
    {
        Warp w{*this, std::mt19937(seed)};
        const Meet meet{&bars};
        const bool leads = warp == 0;
        if (leads && w.wait([&] { return k_full > 0; })) scores[g] = 1;
        bool ok = true;
        int s = 0;
        for (; s < n; ++s) {
            if (!(ok = w.wait([&] { return scores[g] > s; }))) break;
            w.pause();
            if (w.rng() % 3 == 0 && !(ok = w.wait([&] { return values[g] >= s; }))) break;  // sums are rescaled
            if (!leads) {
                meet.arrive<128>(kvl::weights_bar(g, first + s));
                continue;
            }
            const bool more = s + 1 < n;
            if (!(ok = w.wait([&] { return v_full > s; }) && (!more || w.wait([&] { return k_full > s + 1; })))) break;
            meet.wait<128>(kvl::weights_bar(g, first + s));
            if (two && (g == 1 || s > 0)) meet.wait<64>(kvl::turn_bar(g));
            values[g] = s + 1;
            w.pause();
            if (more) scores[g] = s + 2;
            if (two && (g == 0 || more)) meet.arrive<64>(kvl::turn_bar(1 - g));
        }
        if (!ok) kvl::leave_steps(meet, leads, two, g, first, s, n);
    }
};

}  // namespace

int main(int argc, char **argv)
{
    const int trials = argc > 1 ? std::atoi(argv[1]) : 300;
    std::mt19937 rng(7);
    int left = 0;
    for (int i = 0; i < trials; ++i) {
        Trial t;
        t.n = 1 + rng() % 12;
        t.first = rng() % 5;
        t.two = rng() % 4 != 0;
        t.chance = i % 10 == 0 ? 0 : i % 10 < 5 ? 20 : 400;
        std::vector<std::thread> warps;
        warps.emplace_back([&t, s = rng()] { t.convert(s); });
        for (int g = 0; g < (t.two ? 2 : 1); ++g)
            for (int w = 0; w < 4; ++w) warps.emplace_back([&t, g, w, s = rng()] { t.softmax(g, w, s); });
        for (auto &w : warps) w.join();
        for (int id = 0; id < 16; ++id)
            if (t.bars.count[id]) {
                std::printf("barrier %d: %d arrivals left\n", id, t.bars.count[id]);
                return 1;
            }
        left += t.gone;
        if (t.chance == 0 && (t.gone || t.values[0] != t.n)) {
            std::printf("a trial without a failure did not end\n");
            return 1;
        }
    }
    std::printf("meet: ok, %d of %d given up\n", left, trials);
    return left * 4 < trials;  // most of the failures have to have happened
}

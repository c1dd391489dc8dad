// The shares of an attention call (kvl_attend_shares.cuh) on the CPU: jobs of random sizes cut into shares, whose
// CTAs come to their parts in a random order and may give up at any of them.  Every job cut over several
// shares is joined by one of them if all parts came, by none otherwise, and all counters are zero at the end.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#define __host__
#define __device__
#define __forceinline__ inline
#include "kvl_attend_shares.cuh"

struct Part {
    int job;
    uint32_t first, last;  // shares that hold steps of the job
    bool complete;
};

int main()
{
    std::mt19937 rng(3);
    long split = 0, failed = 0;
    for (int trial = 0; trial < 3000; ++trial) {
        const uint32_t cost = 1 + rng() % 8, ctas = 1 + rng() % 152;
        std::vector<uint32_t> start(1, 0), steps;
        for (int j = 0, n = 1 + rng() % 40; j < n; ++j) {
            steps.push_back(1 + rng() % (rng() % 8 ? 40 : 2000));
            start.push_back(start.back() + cost + steps.back());
        }
        const uint32_t total = start.back(), most = (total + cost + 1) / (cost + 2);
        const kvl::Cut cut(total, ctas < most ? ctas : most);
        // each share's parts, as a CTA walks them
        std::vector<std::vector<Part>> parts(cut.shares);
        std::vector<uint32_t> holders(steps.size(), 0);
        uint32_t at = 0;
        for (uint32_t b = 0; b < cut.shares; ++b) {
            uint32_t u = cut.start(b);
            const uint32_t end = cut.start(b + 1);
            if (u != at || end <= u) return std::printf("share %u: %u .. %u, not from %u\n", b, u, end, at), 1;
            at = end;
            for (size_t j = 0; j < steps.size(); ++j) {
                const uint32_t u0 = start[j] + cost, u1 = start[j + 1];  // its steps
                const uint32_t lo = u > u0 ? u : u0, hi = end < u1 ? end : u1;
                if (hi <= lo) continue;
                parts[b].push_back({int(j), cut.share_of(u0), cut.share_of(u1 - 1), lo == u0 && hi == u1});
                ++holders[j];
            }
        }
        if (at != total) return std::printf("the shares end at %u of %u\n", at, total), 1;
        std::vector<uint32_t> counters(cut.shares, 0), next(cut.shares, 0);
        std::vector<int> joined(steps.size(), 0), broken(steps.size(), 0);
        std::vector<uint32_t> gives_up(cut.shares, ~0u), live;
        const uint32_t chance = trial % 3;  // in none, a few or many of the shares
        for (uint32_t b = 0; b < cut.shares; ++b) {
            live.push_back(b);
            if (chance && rng() % (chance == 1 ? 30 : 3) == 0) gives_up[b] = rng() % (parts[b].size() + 1);
        }
        while (!live.empty()) {
            const size_t pick = rng() % live.size();
            const uint32_t b = live[pick], i = next[b]++;
            if (i >= parts[b].size()) {
                live[pick] = live.back();
                live.pop_back();
                continue;
            }
            const Part &p = parts[b][i];
            if (p.complete) continue;
            const bool none = i >= gives_up[b];  // what it gave up at, and all that follows
            if (b < p.first || b > p.last || p.last - p.first + 1 != holders[p.job])
                return std::printf("share %u is not of %u .. %u\n", b, p.first, p.last), 1;
            uint32_t &c = counters[p.first];
            const kvl::Arrival x = kvl::arrival(c, p.last - p.first + 1, none);
            c += none ? 1 + kvl::kNoResult : 1;
            if (x.last) c = 0;
            joined[p.job] += x.join;
            broken[p.job] += none;
        }
        for (uint32_t b = 0; b < cut.shares; ++b)
            if (counters[b]) return std::printf("counter %u left at %#x\n", b, counters[b]), 1;
        for (size_t j = 0; j < steps.size(); ++j) {
            if (holders[j] < 2) continue;
            ++split;
            failed += broken[j] > 0;
            if (joined[j] != (broken[j] ? 0 : 1)) return std::printf("job %zu joined %d times\n", j, joined[j]), 1;
        }
    }
    std::printf("shares: ok, %ld split jobs, %ld of them given up\n", split, failed);
    return split < 1000 || failed < 500 || failed * 2 > split * 3;
}

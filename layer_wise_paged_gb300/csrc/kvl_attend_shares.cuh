// kvl_attend_shares.cuh -- how an attention call's work is cut into equal shares, one a CTA, and how the shares
// of one job find out which of them is the last.  Host code too: a test runs it with CTAs that give up.
#pragma once

#include <cstdint>

namespace kvl {

// `total` units cut into `shares` contiguous parts whose sizes differ by at most one.  Units are counted
// in 32 bits (a call whose units do not fit, some 10^10 tokens, is refused), as 64-bit divisions would
// be the longest part of a small call's start.
struct Cut {
    uint32_t total, shares, size, rest;  // the first `rest` shares hold size + 1 units
    __host__ __device__ __forceinline__ Cut() {}
    __host__ __device__ __forceinline__ Cut(uint32_t t, uint32_t s) : total(t), shares(s), size(t / s), rest(t - t / s * s) {}
    __host__ __device__ __forceinline__ uint32_t start(uint32_t b) const { return b * size + (b < rest ? b : rest); }
    __host__ __device__ __forceinline__ uint32_t share_of(uint32_t u) const
    {
        const uint32_t large = rest * (size + 1);
        return u < large ? u / (size + 1) : rest + (u - large) / size;
    }
};

// A share's part of a job whose result is in the workspace counts as 1 at the job's counter (that of its first
// share), a part that will not come, as its CTA has given up, as 1 + kNoResult.  Either way the share that
// arrives last clears the counter; it joins the parts if all of them are there.  So the counters are zero
// after every call.
constexpr uint32_t kNoResult = 1u << 16;  // above any number of shares

struct Arrival {
    bool last, join;
};

// before: the counter's value before this arrival.
__host__ __device__ __forceinline__ Arrival arrival(uint32_t before, uint32_t parts, bool no_result)
{
    Arrival x;
    x.last = (before & (kNoResult - 1)) + 1 == parts;
    x.join = x.last && before < kNoResult && !no_result;
    return x;
}

}  // namespace kvl

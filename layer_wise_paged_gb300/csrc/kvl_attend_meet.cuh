// kvl_attend_meet.cuh -- the order in which the softmax warps of the tensor-memory attention kernel meet,
// and how they leave when a wait has run out.  Host code too: a test runs it with threads for warps.
#pragma once

namespace kvl {

// Named barriers (0 is __syncthreads).  In each step the four softmax warps of tile g meet at weights_bar(g, .):
// the issuing warp waits there, the others only arrive.  Then, where both tiles have rows, the issuing warps
// take turns: tile 0's waits at turn_bar(0) (from the second step on) and arrives at turn_bar(1) when it has
// issued its products, tile 1's waits at turn_bar(1) and arrives at turn_bar(0) if a step follows.
// Even and odd steps (of all that the CTA has done for the tile) have barriers of their own, as a warp that
// leaves may be a step ahead of the others.
constexpr int kQBar = 5;  // the converting warps, before they load Q
__host__ __device__ constexpr int weights_bar(int g, unsigned step) { return 1 + g + 8 * int(step & 1); }
__host__ __device__ constexpr int turn_bar(int g) { return 3 + g; }

// The meetings of steps s .. n - 1 of a job for a warp that has given up before its first meeting of step s
// (step 0 is the CTA's `first`): every barrier still gets all the arrivals it counts, no more and no fewer, so
// no warp is left waiting.  Also the warps that would only arrive wait here: otherwise one could arrive twice
// at a barrier before another has come to it once.  A step on, that warp would arrive at the other barrier,
// where it waits.
template <typename Meet>
__host__ __device__ __forceinline__ void leave_steps(Meet meet, bool leads, bool two, int g, unsigned first, int s,
                                                     int n)
{
    for (; s < n; ++s) {
        meet.template wait<128>(weights_bar(g, first + s));
        if (!leads || !two) continue;
        if (g == 1 || s > 0) meet.template wait<64>(turn_bar(g));
        if (g == 0 || s + 1 < n) meet.template arrive<64>(turn_bar(1 - g));
    }
}

}  // namespace kvl

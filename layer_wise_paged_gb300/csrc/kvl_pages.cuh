// kvl_pages.cuh -- what the page bookkeeping's kernels share: block-wide prefix sums, the walk over the
// reference counts, host-side checks.
#pragma once

#include "kvl_quant.cuh"

namespace kvl {
namespace {

constexpr int kThreads = 1024;
constexpr int kPerThread = 8;
constexpr int kTile = kThreads * kPerThread;

// Exclusive prefix sum over the CTA's threads (of int, or of two packed in 64 bits); `total` receives the
// sum.  Every thread of the CTA calls it; scratch holds 32 values, and two calls in a row need
// different ones (or a barrier between them).
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *scratch, T &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) scratch[warp] = y;
    __syncthreads();
    T sums = scratch[lane];  // kThreads / 32 = 32 of them: every warp adds them up for itself
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T z = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += z;
    }
    total = __shfl_sync(0xffffffffu, sums, 31);
    const T before = __shfl_sync(0xffffffffu, sums, warp ? warp - 1 : 0);
    return (warp ? before : T(0)) + y - x;
}

// The counts of this thread's kPerThread pages of the tile at `base` (1 past the end).
__device__ __forceinline__ void load_refs(const int32_t *refs, int64_t base, int64_t N, int (&r)[kPerThread])
{
    const int64_t at = base + int64_t(threadIdx.x) * kPerThread;
    if (at + kPerThread <= N && aligned16(refs)) {
#pragma unroll
        for (int i = 0; i < kPerThread / 4; ++i) {
            const int4 q = reinterpret_cast<const int4 *>(refs + at)[i];
            r[4 * i] = q.x; r[4 * i + 1] = q.y; r[4 * i + 2] = q.z; r[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) r[i] = at + i < N ? refs[at + i] : 1;
    }
}

inline kvl_status check_pages(const kvl_pages *p)
{
    if (!p || p->pool_blocks <= 0 || p->pool_blocks > INT32_MAX || p->block_tokens <= 0 || p->n_slots <= 0 ||
        p->n_slots > (1 << 20) || p->table_stride <= 0 || p->table_stride > INT32_MAX)
        return KVL_EINVAL;
    if (!p->tables || !p->lens || !p->refs || !p->pairs || !p->n_pairs) return KVL_EINVAL;
    if (misaligned4(p->tables) || misaligned4(p->lens) || misaligned4(p->refs) || misaligned4(p->n_pairs) ||
        (reinterpret_cast<uintptr_t>(p->pairs) & 7u))
        return KVL_EALIGN;
    return KVL_OK;
}

inline kvl_status check_batch(const kvl_pages *p, int32_t n, const int32_t *x, const int32_t *y, const void *rep)
{
    const kvl_status s = check_pages(p);
    if (s) return s;
    if (n < 0 || n > p->n_slots || (n > 0 && (!x || !y))) return KVL_EINVAL;
    if (misaligned4(x) || misaligned4(y) || bad_report(rep)) return KVL_EALIGN;
    return KVL_OK;
}

}  // namespace
}  // namespace kvl

// kvl_attend.cuh -- what the attention kernels share: arguments, the visible range of a row,
// and how a call's work is cut into equal shares.
//
// Both kernels compute, for a row with scores s_j = sm_scale q.K_j over the visible tokens,
//   x_j = s_j log2(e) + log2(vs_j),  m = max x_j,  w_j = 2^(x_j - m),
//   O = sum w_j codeV_j,  l = sum w_j / vs_j,   out = O / l,   lse = ln(l) + m ln(2),
// with vs_j the V scale of token j's page: w_j 2^m / vs_j is the probability's numerator.  The
// V scale rides in the exponent, so the products take the codes as they are, and w_j lies in
// [0, 1] with 1 at the token that counts most: as a 16-bit half it has 11 significant bits
// wherever it matters (below 2^-14 of the largest weight an absolute error of 2^-25).  The
// maximum, l, O and every score are 32-bit.
//
// Slots come in groups of 16, each within one page (a page whose size is no multiple of 16
// ends in a part of a group), so a group has one K and one V scale and 16 consecutive rows.
#pragma once

#include "kvl_quant.cuh"

namespace kvl {

struct AttendArgs {
    kvl_cache cache;
    kvl_sequences seqs;
    kvl_attention attn;
    int32_t layer;
    int32_t max_rows;  // entries with at most so many rows (fresh tokens x query heads of a KV head) are
                       // attend_rows', the others attend_chunk's
    uint32_t *counters;
    float *parts;      // partial results of rows split over CTAs
    void *report;
};

namespace {

constexpr int kGroup = 16;

// What stands for m in the exponent is a reference, set kHead above a row's largest x so far and moved
// only when an x passes it by kSlack: weights up to 2^14 are halves still, and those below 2^-14 keep
// 2^-25 of a largest weight that is 2^-4 or more.  So a row's sums are rescaled about once.  (With the
// reference at the maximum and a slack of 8, one of the 128 rows that the tensor-memory kernel steps
// together moved in most steps and held the others up for 1,000 cycles.)
constexpr float kSlack = 14.f, kHead = 4.f;

// `total` units cut into `shares` contiguous parts whose sizes differ by at most one.  Units are counted
// in 32 bits (a call whose units do not fit, some 10^10 tokens, is refused), as 64-bit divisions would
// be the longest part of a small call's start.
struct Cut {
    uint32_t total, shares, size, rest;  // the first `rest` shares hold size + 1 units
    __device__ __forceinline__ Cut() {}
    __device__ __forceinline__ Cut(uint32_t t, uint32_t s) : total(t), shares(s), size(t / s), rest(t - t / s * s) {}
    __device__ __forceinline__ uint32_t start(uint32_t b) const { return b * size + min(b, rest); }
    __device__ __forceinline__ uint32_t share_of(uint32_t u) const
    {
        const uint32_t large = rest * (size + 1);
        return u < large ? u / (size + 1) : rest + (u - large) / size;
    }
};
constexpr uint64_t kMostUnits = uint64_t(1) << 31;

// What one batch entry costs: `tiles` row tiles for each KV head, each walking the groups
// [g0, g0 + groups).
struct Cost {
    Entry e;
    int32_t tiles, g0, groups;
};

__device__ __forceinline__ int32_t group_of(int32_t token, int32_t B, int32_t per_block)
{
    const int32_t b = token / B;
    return b * per_block + (token - b * B) / kGroup;
}


// 16 bytes into shared memory; zeros where !ok (src has to be a valid address all the same).
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2^x; -infinity gives 0.
__device__ __forceinline__ float exp2_of(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The V scale of a page as the kernels use it: at least the smallest an append writes (a page
// of zeros whose scale is 0 contributes nothing either way); a NaN stays.
__device__ __forceinline__ float v_scale(float s) { return s < kTinyScale ? kTinyScale : s; }

}  // namespace

size_t attend_rows_part_bytes(int head_dim);  // for each SM
// most: a bound on the rows (as max_rows) of an entry, which chooses the row tile.
kvl_status launch_attend_rows(const AttendArgs &a, int64_t most, int sms, void *stream);
size_t attend_chunk_part_bytes(int head_dim);
kvl_status launch_attend_chunk(const AttendArgs &a, int sms, void *stream);

}  // namespace kvl

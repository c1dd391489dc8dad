// kvl_attend.cuh -- what the attention kernels share: arguments, the visible range of a row,
// and how a call's work is cut into equal shares.
//
// Both kernels compute, for a row with scores s_j = sm_scale q.K_j over the visible tokens,
//   x_j = s_j log2(e) + log2(vs_j),  w_j = 2^(x_j - m),
//   O = sum w_j codeV_j,  l = sum w_j / vs_j,   out = O / l,   lse = ln(l) + m ln(2),
// with vs_j the V scale of token j's page: w_j 2^m / vs_j is the probability's numerator.  The
// V scale rides in the exponent, so the products take the codes as they are.  m is a reference near
// the largest x_j (kHead, kSlack below).  w_j enters its product as a 16-bit half, which the tensor
// cores take with exact halves of the codes: 11 significant bits down to 2^-14, an absolute error of
// 2^-25 below.  The largest w_j of a row is 2^4 or more, so that is 2^-29 of it.  Bfloats would hold
// every weight but with 8 bits.  l sums the weights before they are rounded.  The reference, l, O and
// every score are 32-bit.
//
// Slots come in groups of 16, each within one page (a page whose size is no multiple of 16
// ends in a part of a group), so a group has one K and one V scale and 16 consecutive rows.
#pragma once

#include "kvl_attend_shares.cuh"
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

// The reference m is set kHead above a row's largest x so far, that is below it, and moved only when an x
// passes it by kSlack.  So weights stay below 2^15.5 (a half holds 2^15.99; half a bit is left for the
// rounding of x), the largest is 2^4 or more, and a row's sums are rescaled about once: one of the 128
// rows that the tensor-memory kernel steps together holds the others up for 1,000 cycles.  Both sides
// (512 tokens on 31,232; prompts; us): -4 and 15.5 222.5 348, -4 and 15 224.5 350, -6 and 15 235 361, -8
// and 15 252 385.  With the reference above the largest x (4 and 14: 221.8 346) weights of 2^-21 of the
// largest were lost, and with them up to a fifth of what a long tail gives beside a peak.
constexpr float kSlack = 15.5f, kHead = -4.f;

constexpr uint64_t kMostUnits = uint64_t(1) << 31;  // see Cut

// What one batch entry costs: `tiles` row tiles for each KV head, each walking the groups
// [g0, g0 + groups).
struct Cost {
    Entry e;
    int32_t tiles, g0, groups;
};

// The first token a row at position `pos` sees, j > pos - window.  (A row stands before token 0 where an
// entry has more rows than tokens; window may be as large as an int.)
__device__ __forceinline__ int32_t first_seen(const AttendArgs &a, int32_t pos)
{
    return a.attn.window > 0 ? max(0, max(0, pos) - a.attn.window + 1) : 0;
}

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

// The V scale of a page as the kernels use it.  Up to the smallest that an append writes, i.e. for a page
// of zeros, any positive one gives the same result, and 2^-80 keeps weights and sums in range: a weight
// 2^(x - m) is lost below 2^-126, which a scale of 1e-30 beside one of 2^20 reached at 2^-15 of the
// largest probability, and l, which divides by the scale, stays finite.  A NaN stays.
__device__ __forceinline__ float v_scale(float s) { return s <= kTinyScale ? 0x1p-80f : s; }

}  // namespace

size_t attend_rows_part_bytes(int head_dim);  // for each SM
// most: a bound on the rows (as max_rows) of an entry, which chooses the row tile.
kvl_status launch_attend_rows(const AttendArgs &a, int64_t most, int sms, void *stream);
size_t attend_chunk_part_bytes(int head_dim);
kvl_status launch_attend_chunk(const AttendArgs &a, int sms, void *stream);

}  // namespace kvl

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
    // attention over a shared prefix only
    kvl_shared shared;
    // What the join reads (see kvl_attend_shared.cu): every entry's Sharing; the rows' O and (reference, sum) over their
    // own tokens and, where the few-rows kernel makes them, over the shared ones (`rows` further); or the
    // tensor-memory kernel's job table and parts, parts_most of them.
    int32_t *sharing;
    float *row_o;          // [2][n_rows][n_heads][64, 128 or 256]
    float *row_ml;         // [2][n_rows][n_heads][2]
    int32_t few;           // the few-rows kernel attends the shared tokens too
    int32_t *part_jobs;
    // [0], [1]: 1 if there are results of the first kernel (of the second); [2]: 1 if those of shared tokens are not all
    // there or not where the join looks, so that no entry that shares tokens is written
    int32_t *parts_done;
    float *group_parts;
    int32_t parts_most;
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
    int32_t lo;  // the first token any row sees
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


// Group g of a batch that shares prefixes, as one entry: the shared tokens in the pages of its first sequence, and
// the rows of all of them.  len = 0 for a group that is left out.
__device__ __forceinline__ Entry load_group(const AttendArgs &a, int32_t g, void *rep)
{
    Entry e = {nullptr, 0, 0, 0};
    const int32_t i0 = a.shared.groups[g], i1 = a.shared.groups[g + 1], P = a.shared.tokens[g];
    if (i0 < 0 || i1 < i0 || i1 > a.seqs.n_seq || P < 0) {
        report(rep, KVL_EINVAL, g);
        return e;
    }
    if (i0 == i1 || P == 0) return e;
    const Entry f = load_entry(a.seqs, a.cache.block_tokens, i0, nullptr);  // (its own problems: where it is an entry)
    const int32_t r0 = a.seqs.starts[i0], r1 = a.seqs.starts[i1];
    if (!f.table || r0 < 0 || r1 < r0 || r1 > a.seqs.n_rows) return e;
    if (P > f.len) {
        report(rep, KVL_ERANGE, g);
        return e;
    }
    e.table = f.table;
    e.len = P;
    e.fresh = r1 - r0;
    e.row0 = r0;
    return e;
}

// What an entry shares with the others of its group: its first `tokens` tokens (-1: the entry is left out), its
// group and the group's first row.
struct alignas(16) Sharing {
    int32_t tokens, group, row0, reserved;
};

// Up to kHeldGroups groups as a CTA holds them in shared memory: looked up there, an entry's sharing is a few dozen
// cycles, in memory half a dozen loads one after another.
constexpr int kHeldGroups = 128;
struct HeldGroup {
    int32_t tokens;            // as given
    int32_t len, row0, fresh;  // of load_group
};
struct HeldGroups {
    int32_t first[kHeldGroups + 1];
    HeldGroup group[kHeldGroups];
};

// By a whole CTA, before a barrier.  Whether a group of this thread's ends before it begins.
__device__ __forceinline__ bool hold_groups(const AttendArgs &a, HeldGroups &held)
{
    const int n = a.shared.n_groups;
    const bool here = n <= kHeldGroups;
    bool falls = false;
    if (!here && blockIdx.x > 0) return false;  // (nothing to hold; one CTA looks at the order)
    for (int g = threadIdx.x; g <= n; g += blockDim.x) {
        const int32_t first = a.shared.groups[g];
        if (here) held.first[g] = first;
        if (g == n) continue;
        falls = falls || a.shared.groups[g + 1] < first;
        if (!here) continue;
        const Entry p = load_group(a, g, nullptr);
        held.group[g] = HeldGroup{a.shared.tokens[g], p.len, p.row0, p.fresh};
    }
    return falls;
}

// Entry i, resolved as e; one whose group is left out, or one of whose rows does not see all shared tokens, is left out.
__device__ __forceinline__ Sharing sharing_of(const AttendArgs &a, const HeldGroups &held, const Entry &e, int32_t i, void *rep)
{
    Sharing s = {0, 0, 0, 0};
    const bool here = a.shared.n_groups <= kHeldGroups;
    const int32_t *first = here ? held.first : a.shared.groups;
    int lo = -1, hi = a.shared.n_groups;  // the last group that begins at i or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid;
    }
    if (e.fresh <= 0 || lo < 0 || i >= first[lo + 1]) return s;
    HeldGroup p;
    if (here) {
        p = held.group[lo];
    } else {
        const Entry g = load_group(a, lo, nullptr);
        p = HeldGroup{a.shared.tokens[lo], g.len, g.row0, g.fresh};
    }
    if (p.tokens == 0) return s;
    s.group = lo;
    s.row0 = p.row0;
    s.tokens = p.len;
    if (p.len > 0 && p.len <= e.len - e.fresh && e.row0 >= p.row0 && e.row0 + e.fresh <= p.row0 + p.fresh) return s;
    if (p.len > 0) report(rep, KVL_ERANGE, i);  // (a group reports itself)
    s.tokens = -1;
    return s;
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a group's K tile.  A lane reads it by rows lane/4 and chunks
// lane%4 + 4i; the chunk is XORed so that the 8 lanes of a shared-memory phase hit 8 different
// 16-byte columns of 128.
template <int D>
__device__ __forceinline__ uint32_t k_at(int r, int c)
{
    if constexpr (D == 64) return r * 64 + c * 16;
    else return r * D + ((c ^ ((r & 1) << 2)) << 4);
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
// The parts of attention over a shared prefix: every entry's own tokens, and with a.few the groups' shared ones.
kvl_status launch_attend_row_parts(const AttendArgs &a, int64_t most, int sms, void *stream);
size_t attend_chunk_part_bytes(int head_dim);
constexpr int kChunkJobRows = 256;  // of the tensor-memory kernel's jobs
// The groups' shared tokens.  Its CTAs may start beside the kernel before it on the stream, whose end they wait for.
kvl_status launch_attend_chunk_groups(const AttendArgs &a, int sms, void *stream);
kvl_status launch_attend_chunk(const AttendArgs &a, int sms, void *stream);

// Entries with more rows than this (fresh tokens x query heads of a KV head) go to the tensor-memory kernel.
constexpr int kChunkRows = 40;
// What attention's entry points check alike.  nothing: the call has no work.
kvl_status check_attend(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs, const kvl_attention *attn,
                        const void *d_workspace, size_t workspace_bytes, const void *d_report, bool *nothing);
AttendArgs attend_args(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs, const kvl_attention *attn,
                       void *d_workspace, void *d_report);

}  // namespace kvl

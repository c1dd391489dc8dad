// kvl_evict.cu -- shorten sequences of a cache to the tokens that matter: which stay, where they go, and their
// move into fresh pages.
//
// A sequence of len > keep tokens keeps its first f = min(first, keep), its last r = min(recent, keep - f) and, of
// those between, the keep - f - r with the largest mass (of equals the first).  They keep their order: the k-th of
// them becomes token k.  Pages before f / B stay; from there on the sequence gets fresh pages, so a page that a
// fork still names is never written, sources and destinations are disjoint, and how many pages a batch needs does
// not depend on the masses:
//   plan    one CTA: checks, needs, and the lowest free numbers in batch order (as extend);
//   select  a cluster of CTAs a sequence: the smallest mass that stays by its digits (three passes of 11, 11 and 10
//           bits over order-preserving keys, histograms added up over the cluster), then one walk in token order
//           that gives each kept token its place, moves its mass and notes where its codes come from;
//   move    all layers' codes, a warp 512 bytes of a row's width of one new page.
#include <algorithm>

#include <cooperative_groups.h>

#include "kvl_pages.cuh"

namespace kvl {
namespace {

constexpr int kDigits = 2048;  // 11 bits
// Tokens of a thread in a round (one sequence of 777, 8 of up to 4,096, one of 30,000, one of 128,000: us with 4 20.4, 208,
// 40.8, 173; with 8 21.8, 209, 38.0, 168; with 16 27.1, 213, 45.4, 169).  A table with room for up to
// 8,192 tokens a sequence has one CTA for each.
constexpr int kRun = 8;
constexpr int kMostRanks = 8;  // CTAs of a sequence

// n / d for 0 <= n < 2^31 by one product: the quotient of n and 2^(31 + s) / d rounded up, s = ceil(log2(d)).
struct Divider {
    uint32_t factor;
    int32_t shift, d;
    explicit Divider(int32_t by) : d(by)
    {
        int s = 0;
        while ((int64_t(1) << s) < by) ++s;
        shift = 31 + s;
        factor = uint32_t(((uint64_t(1) << shift) + by - 1) / by);
    }
    Divider() = default;
    __device__ __forceinline__ int32_t operator()(int32_t n) const { return int32_t((uint64_t(uint32_t(n)) * factor) >> shift); }
};

struct EvictArgs {
    kvl_pages p;
    kvl_eviction e;
    kvl_moves m;
    Divider by_block;
    int32_t n;
    const int32_t *slots;
    void *report;
};

// What entry i asks for.
struct Ask {
    int32_t slot, len, keep;
    int32_t stay;   // pages that stay
    int32_t pages;  // fresh ones; 0 where the sequence is not shortened (or shortened to whole pages that stay)
    int32_t error;
    bool cut;
};

__device__ __forceinline__ Ask ask_of(const EvictArgs &a, int i)
{
    const int32_t B = a.p.block_tokens;
    Ask q = {a.slots[i], 0, a.e.keep[i], 0, 0, KVL_OK, false};
    if (q.slot < 0 || q.slot >= a.p.n_slots || q.keep < 0) {
        q.error = KVL_EINVAL;
        return q;
    }
    q.len = a.p.lens[q.slot];
    if (q.len < 0 || ceil_div64(q.len, B) > a.p.table_stride || (a.e.mass && q.len > a.e.tokens)) {
        q.error = KVL_ERANGE;
        return q;
    }
    q.cut = q.len > q.keep;
    q.stay = min(a.e.first, q.keep) / B;
    if (q.cut) q.pages = int32_t(ceil_div64(q.keep, B)) - q.stay;
    return q;
}

// at[i]: where entry i's pages begin in `to`; at[n]: -1 if nothing is done.
__global__ void __launch_bounds__(kThreads) evict_plan_kernel(const __grid_constant__ EvictArgs a)
{
    extern __shared__ uint32_t named[];  // one bit a slot
    __shared__ long long scan_need[32];
    __shared__ int scan_free[32], s_bad;
    const int tid = threadIdx.x;
    allow_dependents_launch();
    for (int w = tid; w < (a.p.n_slots + 31) / 32; w += kThreads) named[w] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    long long need = 0;
    for (int base = 0; base < a.n; base += kThreads) {
        const int i = base + tid;
        Ask q = {};
        if (i < a.n) {
            q = ask_of(a, i);
            if (q.error == KVL_OK && (atomicOr(&named[q.slot >> 5], 1u << (q.slot & 31)) >> (q.slot & 31) & 1u))
                q.error = KVL_EDUP;
            if (q.error) {
                report(a.report, q.error, i);
                s_bad = 1;
            }
        }
        long long total;
        if (base) __syncthreads();  // readers of the scan before
        const long long at = need + block_scan<long long>(q.pages, scan_need, total);
        if (i < a.n) a.m.at[i] = int32_t(min(at, (long long)INT32_MAX));
        need += total;
    }
    __syncthreads();
    bool ok = s_bad == 0 && need <= a.p.pool_blocks;
    if (ok) {
        // are there that many?  (counted before any is taken)
        long long held = 0;
        for (int64_t base = 0; base < a.p.pool_blocks && held < need; base += kTile) {
            int r[kPerThread], mine = 0, total;
            load_refs(a.p.refs, base, a.p.pool_blocks, r);
#pragma unroll
            for (int k = 0; k < kPerThread; ++k) mine += r[k] == 0;
            if (base) __syncthreads();
            block_scan<int>(mine, scan_free, total);
            held += total;
        }
        ok = held >= need;
    }
    if (!ok) {
        if (tid == 0) {
            if (s_bad == 0) report(a.report, KVL_ERANGE, a.n);
            a.m.at[a.n] = -1;
            *a.m.n = 0;
        }
        return;
    }
    long long given = 0;
    for (int64_t base = 0; base < a.p.pool_blocks && given < need; base += kTile) {
        int r[kPerThread], mine = 0, total;
        load_refs(a.p.refs, base, a.p.pool_blocks, r);
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) mine += r[k] == 0;
        __syncthreads();
        long long at = given + block_scan<int>(mine, scan_free, total);
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            if (r[k] != 0) continue;
            if (at < need) {
                const int64_t id = base + int64_t(tid) * kPerThread + k;
                a.m.to[at] = int32_t(id);
                a.p.refs[id] = 1;
            }
            ++at;
        }
        given += total;
    }
    if (tid == 0) {
        a.m.at[a.n] = int32_t(need);
        *a.m.n = int32_t(need);
    }
}

// Larger keys are larger masses; -0 is 0, and a NaN comes last.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (x != x) return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A cluster of CTAs a sequence: a thread holds kRun tokens' masses in registers, so a sequence of up to kRun * 1024
// tokens a CTA is read once (longer ones again for every pass, in rounds).
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictArgs a)
{
    __shared__ uint32_t hist[2][kDigits];
    __shared__ long long scan[32];
    __shared__ int scan_bins[32];
    __shared__ uint32_t s_digit, s_rest;
    __shared__ uint32_t s_count[kRun * 32];  // of a round's 32 tokens: those that surely stay, those of the least mass << 16
    __shared__ uint32_t s_before[kRun * 32];
    __shared__ long long s_total;
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = int(cluster.num_blocks()), rank = int(cluster.block_rank()), i = blockIdx.x / ranks;
    allow_dependents_launch();
    // (the choice needs nothing of the plan, which runs meanwhile; an entry that the plan refuses is not acted on)
    const Ask q = ask_of(a, i);
    if (q.error || !q.cut) {
        grid_dependency_wait();  // the plan has ended when this kernel has
        return;
    }
    const int32_t B = a.p.block_tokens;
    const int f = min(a.e.first, q.keep), r = min(a.e.recent, q.keep - f);
    const int lo = f, hi = q.len - r;       // the tokens to choose from
    const int take = q.keep - f - r;        // how many of them stay; fewer than there are
    float *mass = a.e.mass ? a.e.mass + int64_t(q.slot) * a.e.mass_stride : nullptr;
    int32_t *table = a.p.tables + int64_t(q.slot) * a.p.table_stride;
    // Token of a round's slot y; slots from `live` on hold none (of any thread).  (A sequence's end and a round fit 32 bits
    // without a sign.)
    const uint32_t round = uint32_t(ranks) * kThreads * kRun, len = uint32_t(q.len);
    const int rounds = int((len - 1) / round) + 1;
    float x[kRun];
    auto first_of = [&](int n) { return n * round + uint32_t(rank) * (kRun * kThreads); };
    auto live_of = [&](int n) { return first_of(n) < len ? int((len - first_of(n) - 1) / kThreads) + 1 : 0; };
    auto load = [&](int n) {
        const int live = live_of(n);
#pragma unroll
        for (int y = 0; y < kRun; ++y) {
            x[y] = 0.f;
            if (y < live) {
                const uint32_t j = first_of(n) + y * kThreads + tid;
                if (mass && j < len) x[y] = __ldcg(mass + j);
            }
        }
    };
    load(0);

    // ---- the smallest key that stays, and how many of those that equal it
    uint32_t least = 0xffffffffu, equals = 0;
    if (take > 0 && !mass) {
        least = key_of(0.f);
        equals = take;
    } else if (take > 0) {
        uint32_t known = 0, mask = 0, rest = take;  // the key's digits so far; its rank among those that have them
        for (int z = tid; z < kDigits; z += kThreads) hist[0][z] = 0;
        __syncthreads();
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            uint32_t *mine = hist[pass & 1];
#pragma unroll 1
            for (int n = 0; n < rounds; ++n) {
                if (rounds > 1) load(n);
                const int live = live_of(n);
#pragma unroll
                for (int y = 0; y < kRun; ++y) {
                    if (y >= live) continue;
                    const uint32_t j = first_of(n) + y * kThreads + tid, k = key_of(x[y]);
                    if (j >= uint32_t(lo) && j < uint32_t(hi) && (k & mask) == known) atomicAdd(&mine[(k >> shift) & (bins - 1)], 1u);
                }
            }
            cluster.sync();
            // the digit at which the sum from the largest digit down reaches `rest`: two bins a thread
            const int top = bins - 1 - 2 * tid;
            int c0 = 0, c1 = 0;
            if (2 * tid < bins)
                for (int z = 0; z < ranks; ++z) {
                    const uint32_t *theirs = cluster.map_shared_rank(mine, z);
                    c0 += theirs[top];
                    c1 += theirs[top - 1];
                }
            for (int z = tid; z < kDigits; z += kThreads) hist[~pass & 1][z] = 0;  // (its readers have passed)
            int total;
            const uint32_t before = block_scan<int>(c0 + c1, scan_bins, total);
            if (before < rest && rest <= before + c0) {
                s_digit = top;
                s_rest = rest - before;
            } else if (before + c0 < rest && rest <= before + c0 + c1) {
                s_digit = top - 1;
                s_rest = rest - before - c0;
            }
            __syncthreads();
            known |= s_digit << shift;
            mask |= uint32_t(bins - 1) << shift;
            rest = s_rest;
            __syncthreads();
        }
        least = known;
        equals = rest;
    }

    // ---- places, masses, sources.  A round's masses are in registers before any is written, and a token moves down,
    // never past tokens that a later round still reads.
    grid_dependency_wait();
    if (a.m.at[a.n] < 0) {  // refused
        cluster.sync();     // (the others may still be reading this CTA's histogram)
        return;
    }
    const int64_t first_page = a.m.at[i];
    long long kept = 0;  // tokens that stay before this round; those that equal `least` in the high half
#pragma unroll 1
    for (int n = 0; n < rounds; ++n) {
        if (rounds > 1) load(n);
        const int live = live_of(n);
        unsigned sure[kRun], even[kRun];
#pragma unroll
        for (int y = 0; y < kRun; ++y) {
            sure[y] = even[y] = 0;
            if (y >= live) {
                if (lane == 0) s_count[y * 32 + warp] = 0;
                continue;
            }
            const uint32_t j = first_of(n) + y * kThreads + tid, k = key_of(x[y]);
            const bool between = j >= uint32_t(lo) && j < uint32_t(hi);
            sure[y] = __ballot_sync(0xffffffffu, j < len && (!between || (take > 0 && k > least)));
            even[y] = __ballot_sync(0xffffffffu, between && take > 0 && k == least);
            if (lane == 0) s_count[y * 32 + warp] = __popc(sure[y]) | __popc(even[y]) << 16;
        }
        __syncthreads();
        const uint32_t c = tid < kRun * 32 ? s_count[tid] : 0;
        long long total;
        const long long b = block_scan<long long>((c & 0xffffu) | (long long)(c >> 16) << 32, scan, total);
        if (tid < kRun * 32) s_before[tid] = uint32_t(b & 0xffff) | uint32_t(b >> 32) << 16;  // (each at most kRun * 1,024)
        if (tid == 0) s_total = total;
        cluster.sync();
        long long all = 0, ahead = kept;
        for (int z = 0; z < ranks; ++z) {
            const long long t = *cluster.map_shared_rank(&s_total, z);
            all += t;
            if (z < rank) ahead += t;
        }
        kept += all;
#pragma unroll
        for (int y = 0; y < kRun; ++y) {
            if (y >= live) continue;
            const uint32_t w = s_before[y * 32 + warp], below = (1u << lane) - 1;
            const int s = int(ahead & 0xffffffffll) + int(w & 0xffffu) + __popc(sure[y] & below);
            const int v = int(ahead >> 32) + int(w >> 16) + __popc(even[y] & below);
            const bool stays = sure[y] >> lane & 1u, equal = even[y] >> lane & 1u;
            if (stays || (equal && v < int(equals))) {
                const int j = int(first_of(n) + y * kThreads + tid), k = s + min(v, int(equals)), k_blk = a.by_block(k), at = k_blk - q.stay;
                if (mass) mass[k] = x[y];
                if (at >= 0) {
                    const int j_blk = a.by_block(j);
                    const int32_t page = table[j_blk];
                    const bool there = page >= 0 && page < a.p.pool_blocks;
                    if (!there) report(a.report, KVL_ERANGE, i);
                    reinterpret_cast<int2 *>(a.m.from)[(first_page + at) * B + k - k_blk * B] = make_int2(there ? page : -1, j - j_blk * B);
                }
            }
        }
        cluster.sync();  // the sums, and the masses
    }
    const int me = rank * kThreads + tid, all = ranks * kThreads;
    if (mass)
        for (int64_t j = q.keep + me; j < a.e.tokens; j += all) mass[j] = 0.f;
    const int pages = int(ceil_div64(q.keep, B));
    for (int64_t k = q.keep + me; k < int64_t(pages) * B; k += all)
        if (q.pages > 0) reinterpret_cast<int2 *>(a.m.from)[(first_page + k / B - q.stay) * B + k % B] = make_int2(-1, 0);
    // ---- the pages that go
    const int held = int(ceil_div64(q.len, B));
    for (int k = q.stay + me; k < held; k += all) {
        const int32_t id = table[k];
        if (id < 0 || id >= a.p.pool_blocks) {
            report(a.report, KVL_ERANGE, i);
        } else if (atomicSub(&a.p.refs[id], 1) <= 0) {
            atomicAdd(&a.p.refs[id], 1);
            report(a.report, KVL_EINVAL, i);
        }
    }
    cluster.sync();
    for (int k = q.stay + me; k < pages; k += all) table[k] = a.m.to[first_page + k - q.stay];
    if (me == 0) a.p.lens[q.slot] = q.keep;
}

// ---- codes -------------------------------------------------------------------------------------

// (8 prompts to 1,024 tokens, 32 layers, plan and selection with it: 210 us; measured beside each other three CTAs an SM
// 224, four, which spill, 268, six of half the tokens on their way 306.  The moves alone, pages of 16 / 64: e4m3 190 / 208,
// int8 215 / 236: a page of 64 has four parts of two slices, each of which looks at all its scales)
constexpr int kMoveThreads = 256, kMoveCtasPerSm = 3;
constexpr int kHeld = 8;  // tokens whose codes a lane has on their way

struct MoveArgs {
    kvl_cache c;
    kvl_moves m;
    int64_t max_pages;
    int32_t lanes;   // lanes of a row's slice: a power of two, 16 bytes each
    int32_t slices;  // of a row of H * d bytes
    int32_t parts;   // of a page's slots, `part` slots (at most 32) each
    int32_t part;
    void *report;
};

// round(code * ratio) of four codes, 0 <= ratio <= 1, the product rounded to 32 bits first.
template <int CODE>
__device__ __forceinline__ uint32_t turn4(uint32_t w, float ratio)
{
    if constexpr (CODE == KVL_CODE_FLOAT) {
        uint32_t l, g;
        codes_of<CODE>(w, l, g);
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&l)), q = __half22float2(*reinterpret_cast<const __half2 *>(&g));
        return to_codes4<CODE>(p.x * ratio, p.y * ratio, q.x * ratio, q.y * ratio);
    } else {
        // A code c is read as the float 2^23 + (c + 128), of which 2^23 + 128 is taken; adding 1.5 * 2^23 rounds the
        // product to a whole number, which is the sum's lowest byte.  (Products stay within a code's range.)
        const uint32_t x = w ^ 0x80808080u;
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = __uint_as_float(__byte_perm(x, 0x4b000000u, 0x7650 | i)) - 8388736.f;
            r[i] = __float_as_uint(__fadd_rn(__fmul_rn(c, ratio), 12582912.f));
        }
        return __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
    }
}

// scale' = the largest scale of the pages that a new page's tokens come from, for each head; code' =
// round(code * (scale / scale')).  The tokens of the largest scale keep their codes bit for bit, so what a further
// eviction rounds again is what came from smaller ones.  A warp takes a part of a page's slots (all of whose scales
// it looks at) and a slice of their rows; the next unit's sources and this one's codes are on their way while the
// scales are looked at.
template <int CODE>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtasPerSm) move_tokens_kernel(const __grid_constant__ MoveArgs a)
{
    grid_dependency_wait();
    int64_t n = *a.m.n;
    if (n < 0 || n > a.max_pages) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.report, KVL_ERANGE, n);
        n = n < 0 ? 0 : a.max_pages;
    }
    const int64_t N = a.c.pool_blocks, planes = int64_t(a.c.n_layers) * 2;
    const int B = a.c.block_tokens, H = a.c.n_kv_heads, d = a.c.head_dim, row_bytes = H * d;
    const int lane = threadIdx.x & 31, per = 32 / a.lanes, rw = lane / a.lanes, ch = lane % a.lanes;
    const uint32_t per_plane = uint32_t(a.slices) * a.parts, per_page = uint32_t(planes) * per_plane;  // (the host has checked)
    const int64_t units = n * per_page, step = int64_t(gridDim.x) * (kMoveThreads / 32);

    // A unit: part of page k (its fresh page, lane l's source there), plane and slice.
    struct Unit {
        int64_t k;
        uint32_t lp;
        int slice, s_first, to;
        int2 from;
    };
    auto source = [&](int64_t k, int slot) -> int2 {  // page and slot, a page of -1: none
        const int2 x = slot < B ? reinterpret_cast<const int2 *>(a.m.from)[k * B + slot] : make_int2(-1, 0);
        return make_int2(x.x < N && x.y >= 0 && x.y < B ? x.x : -1, x.y);
    };
    auto unit_at = [&](int64_t u) {
        Unit x;
        x.k = u / per_page;
        uint32_t rest = uint32_t(u - x.k * per_page);
        x.lp = rest / per_plane;
        rest -= x.lp * per_plane;
        x.slice = int(rest / uint32_t(a.parts));
        x.s_first = int(rest - uint32_t(x.slice) * a.parts) * a.part;
        x.to = a.m.to[x.k];
        x.from = source(x.k, lane < a.part ? x.s_first + lane : B);
        return x;
    };
    int64_t u = int64_t(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5);
    if (u >= units) return;
    Unit next = unit_at(u);
    for (; u < units; u += step) {
        const Unit x = next;
        if (u + step < units) next = unit_at(u + step);
        const int first = x.slice * a.lanes * 16, at = first + ch * 16;  // the slice's bytes of a row, and this lane's
        const bool mine = at < row_bytes;
        if (x.to < 0 || x.to >= N) {
            if (lane == 0) report(a.report, KVL_ERANGE, x.k);
            continue;
        }
        const int h = mine ? at / d : 0, ha = first / d, hb = (min(first + a.lanes * 16, row_bytes) - 1) / d;  // heads of the slice
        const uint8_t *codes = static_cast<const uint8_t *>(a.c.codes) + x.lp * N * B * row_bytes + (mine ? at : 0);
        uint8_t *dst = static_cast<uint8_t *>(a.c.codes) + ((int64_t(x.lp) * N + x.to) * B + x.s_first) * row_bytes + (mine ? at : 0);
        const float *scales = a.c.scales + x.lp * N * H;
        uint4 w[kHeld];
        float was[kHeld];
        auto load = [&](int s0) {  // slots s0 + rw, s0 + per + rw, ... of the part
#pragma unroll
            for (int y = 0; y < kHeld; ++y) {
                const int s = s0 + y * per + rw;
                const int32_t page = __shfl_sync(0xffffffffu, x.from.x, s & 31), slot = __shfl_sync(0xffffffffu, x.from.y, s & 31);
                was[y] = -1.f;  // none
                if (s < a.part && page >= 0 && mine) {
                    w[y] = *reinterpret_cast<const uint4 *>(codes + (int64_t(page) * B + slot) * row_bytes);
                    was[y] = scales[int64_t(page) * H + h];
                }
            }
        };
        load(0);
        // lane l looks at the scales of tokens l, l + 32, ... for each head of the slice
        float now = 0.f;
        for (int s = 0; s < B; s += 32) {
            const int32_t page = a.parts == 1 ? x.from.x : source(x.k, s + lane).x;
#pragma unroll 4
            for (int y = ha; y <= hb; ++y) {
                const float v = page >= 0 ? scales[int64_t(page) * H + y] : 0.f;
                const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, v > 0.f ? __float_as_uint(v) : 0u));
                if (y == h) now = fmaxf(now, top);
            }
        }
        for (int s0 = 0; s0 < a.part; s0 += per * kHeld) {
            if (s0 > 0) load(s0);
#pragma unroll
            for (int y = 0; y < kHeld; ++y) {
                if (was[y] == -1.f) continue;
                if (was[y] != now) {
                    const float ratio = __fdiv_rn(was[y], now);
                    w[y] = make_uint4(turn4<CODE>(w[y].x, ratio), turn4<CODE>(w[y].y, ratio), turn4<CODE>(w[y].z, ratio),
                                      turn4<CODE>(w[y].w, ratio));
                }
                *reinterpret_cast<uint4 *>(dst + int64_t(s0 + y * per + rw) * row_bytes) = w[y];
            }
        }
        if (x.s_first == 0 && mine && rw == 0 && at % d == 0) a.c.scales[(int64_t(x.lp) * N + x.to) * H + h] = now;
    }
}

inline kvl_status check_moves(const kvl_moves *m)
{
    if (!m || !m->from || !m->to || !m->at || !m->n) return KVL_EINVAL;
    if ((reinterpret_cast<uintptr_t>(m->from) & 7u) || misaligned4(m->to) || misaligned4(m->at) || misaligned4(m->n))
        return KVL_EALIGN;
    return KVL_OK;
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" kvl_status kvl_pages_evict(const kvl_pages *pages, int32_t n, const int32_t *slots,
                                      const kvl_eviction *eviction, const kvl_moves *moves, void *d_report, void *stream)
{
    if (!eviction) return KVL_EINVAL;
    kvl_status s = check_batch(pages, n, slots, eviction->keep, d_report);
    if (!s) s = check_moves(moves);
    if (s) return s;
    if (eviction->first < 0 || eviction->recent < 0 || (eviction->mass && (eviction->tokens <= 0 || eviction->mass_stride < eviction->tokens))) return KVL_EINVAL;
    if (misaligned4(eviction->mass)) return KVL_EALIGN;
    EvictArgs a;
    a.p = *pages;
    a.e = *eviction;
    a.m = *moves;
    a.by_block = Divider(pages->block_tokens);
    a.n = n;
    a.slots = slots;
    a.report = d_report;
    static std::atomic<unsigned long long> ready[kMaxDevices];
    const int smem = (pages->n_slots + 31) / 32 * 4;
    if (smem > 32 * 1024 && !allow_smem(evict_plan_kernel, ready, (1 << 20) / 8)) return KVL_ECUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    evict_plan_kernel<<<1, kThreads, smem, st>>>(a);
    s = launch_status();
    if (s || n == 0) return s;
    // as many CTAs a sequence as hold the longest that the table has room for in their registers
    const int64_t most = std::min(pages->table_stride * int64_t(pages->block_tokens), pages->pool_blocks * int64_t(pages->block_tokens));
    unsigned ranks = 1;
    while (ranks < kMostRanks && int64_t(ranks) * kThreads * kRun < most) ranks *= 2;
    return launch_behind(evict_select_kernel, unsigned(n) * ranks, kThreads, 0, stream, a, ranks);
}

extern "C" kvl_status kvl_tokens_move(const kvl_cache *cache, const kvl_moves *moves, int64_t max_pages,
                                      void *d_report, void *stream)
{
    kvl_status s = check_cache(cache);
    if (!s && (max_pages < 0 || max_pages > INT32_MAX)) s = KVL_EINVAL;
    if (s || max_pages == 0) return s;
    if ((s = check_moves(moves))) return s;
    if (bad_report(d_report)) return KVL_EALIGN;
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    MoveArgs a;
    a.c = *cache;
    a.m = *moves;
    a.max_pages = max_pages;
    const int vectors = cache->n_kv_heads * cache->head_dim / 16;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < vectors) a.lanes *= 2;
    a.slices = (vectors + a.lanes - 1) / a.lanes;
    a.part = std::min(2 * kHeld * (32 / a.lanes), 32);
    a.parts = int32_t((int64_t(cache->block_tokens) + a.part - 1) / a.part);
    if (int64_t(cache->n_layers) * 2 * a.slices * a.parts > INT32_MAX) return KVL_EINVAL;
    a.report = d_report;
    const int ctas = sms * kMoveCtasPerSm;
    return launch_behind(cache->code_type == KVL_CODE_FLOAT ? move_tokens_kernel<KVL_CODE_FLOAT> : move_tokens_kernel<KVL_CODE_INT>,
                         ctas, kMoveThreads, 0, stream, a);
}

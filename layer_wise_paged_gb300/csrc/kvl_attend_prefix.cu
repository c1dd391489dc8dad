// kvl_attend_prefix.cu -- attention of a group's rows over the tokens its sequences share, on the tensor cores.
//
// The rows of a group (its sequences' fresh tokens times the query heads of a KV head) are a few dozen to a few
// hundred, and each shared byte should be read and converted for as many of them as possible while the products
// stay below the time that reading takes.  So tokens fill the 128-high operand and up to 128 rows the other:
//   S^T [128 tokens x rows] = K Q^T,   O^T [head_dim x rows] += V^T P^T,
// where rows in the high operand would pad 30 of them to 128.  A thread of the softmax holds one token and 32 rows at
// a time: its weights go to shared memory as halves, as the second product's operand (over the step's K, which is
// done with); a row's sum stays in the threads' registers and is added up over the tokens once a job, and the rows'
// references (kvl_attend.cuh) are looked at by one vote, moved only when a score has outgrown its own.
//   warps 0-3, 4-7   softmax of the first and second 32 of each 64 rows; lanes of tensor memory are tokens, then
//                    elements of O
//   warps 8-11       read the codes of a step's 8 groups, two each, and convert them to halves (exact); the rows
//   warp 12          issues the products: S^T of the step to come, then O^T of the step whose weights are there
// A (group, KV head, tile of rows) is a job of as many steps of 128 slots as its tokens need; the steps of all jobs in
// a row are cut into equal contiguous shares, one a CTA.  Every share's part of a job goes to memory, and whoever
// reads the results (the kernel over the sequences' own tokens) adds the parts up in the order of the shares.
//
// Every wait is bounded.  Past the limit a flag is raised and no wait waits any longer, but every warp goes through
// all its steps and barriers, so none is left behind; nothing is written and the report says KVL_ETIMEOUT.
#include "kvl_attend_prefix.cuh"
#include "kvl_tcgen.cuh"

namespace kvl {
namespace {

constexpr int kSlots = 128;               // of a step
constexpr int kGroups = kSlots / kGroup;  // 8
constexpr int kSoftmax = 8;               // warps
constexpr int kWarps = kSoftmax + 4 + 1;  // 128 registers a thread
constexpr int kThreads = kWarps * 32;
constexpr int kPlaces = 4;                // steps whose scales are kept: the softmax may be two behind the conversion
constexpr int kKStages = 2;               // K's, which hold the step's weights later, and V's
constexpr int kVStages = 2;
// Units of a share: a job's steps, and kJobCost before them for loading its rows and writing its part.
constexpr int kJobCost = 4;
constexpr int kUnitsPerCta = kJobCost + 2;
constexpr float kNoScore = -1e30f;        // a row's reference before its first score

struct alignas(16) Places {
    float ks[kGroups], lvs[kGroups], ivs[kGroups];
    int32_t nv[kGroups];
};

constexpr int ROWS = kPrefixTileRows;     // of a tile: 32 a softmax thread
static_assert(ROWS == 64, "two softmax warpgroups of 32 rows each");

template <int D>
struct Prefix {
    static constexpr int kVBytes = kSlots * D * 2;
    static constexpr int kPBytes = kSlots * 128;
    static constexpr int kKBytes = kVBytes > kPBytes ? kVBytes : kPBytes;
    static constexpr int kQBytes = ROWS * D * 2;
    static constexpr int kV = 0;  // (at head_dim 64 the 128-high operand's second half reads on behind V: never past K)
    static constexpr int kQ = kV + kVStages * kVBytes;
    static constexpr int kK = kQ + kQBytes;
    // K or V codes of a step, on their way: 16 KB each at head_dim 128 (with the step ahead in registers instead
    // 3.0 us a step of 128 rows, 2.4 of 64: the reads' latency)
    static constexpr int kUnitBytes = kSlots * D;
    static constexpr int kUnits = D == 64 ? 8 : 4;
    static constexpr int kRing = kK + kKStages * kKBytes;
    static constexpr int kSmem = kRing + kUnits * kUnitBytes + 1024;
};

// P_FULL and PV_DONE come in pairs, for even and odd steps, as a softmax warp may be a step ahead of the products: its
// weights of step k + 1 may be there before the products have looked for those of step k.  Of one barrier two phases
// would have passed then, and a wait for the first would never end (or, for PV_DONE, end too early).
enum Bar { K_FULL = 0, K_EMPTY = 2, V_FULL = 4, V_EMPTY = 6, S_FULL = 8, P_FULL = 10, PV_DONE = 12, Q_FULL = 14, LEAVE = 15, BARS = 16 };

// A group as a batch of jobs.
struct Shared {
    Entry e;             // its tokens, and all its rows
    int32_t tiles, steps;
};

__device__ __forceinline__ Shared shared_at(const AttendArgs &a, int g, void *rep)
{
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup;
    Shared s;
    s.e = load_group(a, g, rep);
    s.tiles = s.e.len > 0 ? int32_t((int64_t(s.e.fresh) * (a.attn.n_heads / a.cache.n_kv_heads) + ROWS - 1) / ROWS) : 0;
    s.steps = s.e.len > 0 ? (group_of(s.e.len - 1, B, per_block) + kGroups) / kGroups : 0;
    return s;
}

// A walk over the jobs of a share, each role's own.
struct Walk {
    uint32_t u, u_end;
    int32_t group, job, before;  // job of the group; jobs of the groups before it
    Shared s;
    int32_t h, tile, sa, n;      // KV head, tile of rows, steps [sa, sa + n)
    uint32_t u0;                 // the unit of the job's first step
    uint32_t taken;

    __device__ __forceinline__ void here(uint32_t in)  // u is the in-th unit of the job
    {
        h = job / s.tiles;
        tile = job - h * s.tiles;
        taken = min(uint32_t(s.steps + kJobCost) - in, u_end - u);
        sa = max(0, int(in) - kJobCost);
        n = max(0, int(in + taken) - kJobCost) - sa;
        u0 = u - in + kJobCost;
    }
    __device__ __forceinline__ void begin(const AttendArgs &a, uint32_t first, uint32_t end, int g, uint32_t off, int jobs)
    {
        u = first;
        u_end = end;
        group = g;
        before = jobs;
        s = shared_at(a, g, nullptr);
        job = int(off / uint32_t(s.steps + kJobCost));
        here(off - job * uint32_t(s.steps + kJobCost));
    }
    __device__ __forceinline__ bool next(const AttendArgs &a)
    {
        u += taken;
        if (u >= u_end) return false;
        if (++job >= a.cache.n_kv_heads * s.tiles) {
            before += job;
            job = 0;
            do s = shared_at(a, ++group, nullptr); while (s.tiles == 0);
        }
        here(0);
        return true;
    }
};

template <int CODE, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_prefix_kernel(const __grid_constant__ AttendArgs a)
{
    using C = Prefix<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long bars[BARS];
    __shared__ Places places[kPlaces];
    __shared__ __align__(16) float s_refs[2][ROWS];  // of two jobs: the rows' references, negated
    __shared__ float s_factor[2], s_most[4];         // the factor of their scores
    __shared__ float s_join[2][4][32];
    __shared__ uint64_t s_scan[kWarps], s_jobs[kWarps];
    __shared__ uint32_t s_off, s_tmem;
    __shared__ int s_group, s_before, s_gone;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int G = a.attn.n_heads / H, per_block = (B + kGroup - 1) / kGroup;
    const int64_t N = a.cache.pool_blocks, plane = int64_t(a.layer) * 2 * N;

    allow_dependents_launch();
    resolve_entries(a, int(blockIdx.x) * kThreads + tid, int(gridDim.x) * kThreads);
    // ---- this CTA's share of the units, and how many jobs come before it
    const int n_groups = a.shared.n_groups, per_thread = (n_groups + kThreads - 1) / kThreads;
    const int i0 = min(n_groups, tid * per_thread), i1 = min(n_groups, i0 + per_thread);
    uint64_t units = 0, jobs = 0;
    for (int i = i0; i < i1; ++i) {
        const Shared s = shared_at(a, i, blockIdx.x == 0 ? a.report : nullptr);
        units += uint64_t(H) * s.tiles * (s.steps + kJobCost);
        jobs += uint64_t(H) * s.tiles;
    }
    uint64_t scan = units, scan_j = jobs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, scan, o), y = __shfl_up_sync(0xffffffffu, scan_j, o);
        if (lane >= o) {
            scan += x;
            scan_j += y;
        }
    }
    if (lane == 31) {
        s_scan[warp] = scan;
        s_jobs[warp] = scan_j;
    }
    __syncthreads();
    uint64_t before = scan - units, jobs_before = scan_j - jobs, total = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            before += s_scan[w];
            jobs_before += s_jobs[w];
        }
        total += s_scan[w];
    }
    if (blockIdx.x == 0 && tid == 0) *a.shared_done = total < kMostUnits;
    if (total == 0 || total >= kMostUnits) {
        if (total && blockIdx.x == 0 && tid == 0) report(a.report, KVL_ERANGE, n_groups);
        return;
    }
    const Cut cut(uint32_t(total), min(gridDim.x, (uint32_t(total) + kUnitsPerCta - 1) / kUnitsPerCta));
    if (blockIdx.x >= cut.shares) return;
    const uint32_t first = cut.start(blockIdx.x);
    if (first >= before && first < before + units) {
        uint64_t at = before, j = jobs_before;
        int i = i0;
        for (;; ++i) {
            const Shared s = shared_at(a, i, nullptr);
            const uint64_t n = uint64_t(H) * s.tiles * (s.steps + kJobCost);
            if (first < at + n) break;
            at += n;
            j += uint64_t(H) * s.tiles;
        }
        s_group = i;
        s_off = uint32_t(first - at);
        s_before = int(j);
    }

    const uint32_t bar = smem_u32(bars);
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sm = smem_u32(smem);
    if (tid == 0) {
        for (int x = 0; x < kKStages; ++x) {
            mbar_init(bar + 8 * (K_FULL + x), 4);   // the converting warps
            mbar_init(bar + 8 * (K_EMPTY + x), 1);  // O^T of the step
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar + 8 * (V_FULL + x), 4);
            mbar_init(bar + 8 * (V_EMPTY + x), 1);
            mbar_init(bar + 8 * (S_FULL + x), 2);   // S^T, and the issuing thread, by which places and factors reach the softmax
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar + 8 * (P_FULL + x), kSoftmax);
            mbar_init(bar + 8 * (PV_DONE + x), 1);
        }
        mbar_init(bar + 8 * Q_FULL, 4);
        mbar_init(bar + 8 * LEAVE, 1);
        fence_mbar_init();
        s_gone = 0;
    }
    if (warp == kWarps - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem;  // columns: S^T 0 and ROWS, O^T 2 ROWS
    volatile int *gone = &s_gone;
    auto wait = [&](int which, uint32_t parity) {
        const uint32_t at = bar + 8 * which;
        if (!mbar_try_wait(at, parity) && !*gone) wait_bar(at, parity, gone);
        __syncwarp();
    };
    Walk job;
    job.begin(a, first, cut.start(blockIdx.x + 1), s_group, s_off, s_before);
    uint32_t it = 0, jobs_done = 0;  // steps and jobs of this CTA so far: the barriers' phases

    if (warp < kSoftmax) {
        // ---- softmax: token `slot` of a step, rows 64 p + 32 w .. in pass p; its quarter of tensor memory's lanes
        const int w = warp >> 2, quarter = warp & 3, slot = quarter * 32 + lane;
        const uint32_t lanes = tmem + (uint32_t(quarter) << 21) + 32 * w;
        auto meet = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory"); };
        // 32 values of a lane each combined over the warp's lanes: lane l gets that of value l
        auto over_lanes = [&](float (&x)[32], auto join) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const bool up = lane & o;
                    const float send = up ? x[i] : x[i + o], keep = up ? x[i + o] : x[i];
                    x[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
                }
            return x[0];
        };
        do {
            if (job.n == 0) continue;
            float *refs = s_refs[jobs_done & 1] + 32 * w;
            uint64_t l[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) l[i] = 0;
            for (int s = 0; s < job.n; ++s) {
                const uint32_t k = it + s, set = k & 1;
                wait(S_FULL + set, (k >> 1) & 1);
                tmem_fence_after();
                const Places &pl = places[k % kPlaces];
                const int gi = slot / kGroup;
                const bool there = slot % kGroup < pl.nv[gi];
                const float f = pl.ks[gi] * s_factor[jobs_done & 1], lvs = there ? pl.lvs[gi] : -INFINITY, iv = there ? pl.ivs[gi] : 0.f;
                const uint64_t ff = pair_of(f, f), ll = pair_of(lvs, lvs), ii = pair_of(iv, iv);
                const uint32_t ts = lanes + set * ROWS, to = lanes + 2 * ROWS;
                uint32_t v[32];
                // exponents against the rows' references, and whether one has outgrown its own
                auto exponents = [&] {
                    tmem_ld32(ts, v);
                    tmem_wait_ld();
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(refs + i);
                        const float2 y = split_pair(add_pair(fma_pair(pair_of(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), ff, pair_of(m.x, m.y)), ll));
                        const float2 z = split_pair(add_pair(fma_pair(pair_of(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])), ff, pair_of(m.z, m.w)), ll));
                        v[i] = __float_as_uint(y.x);
                        v[i + 1] = __float_as_uint(y.y);
                        v[i + 2] = __float_as_uint(z.x);
                        v[i + 3] = __float_as_uint(z.y);
                        top = max3(max3(top, y.x, y.y), z.x, z.y);
                    }
                    return top > kSlack;
                };
                uint32_t grew;
                asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                             : "=r"(grew)
                             : "r"(uint32_t(exponents())), "r"(1 + w)
                             : "memory");
                if (grew) {
                    // the step's largest x of each row, over all tokens; row `lane` of the 32 is this lane's
                    float x[32];
                    tmem_ld32(ts, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = there ? fmaf(__uint_as_float(v[i]), f, lvs) : -INFINITY;
                    s_join[w][quarter][lane] = over_lanes(x, [](float y, float z) { return fmaxf(y, z); });
                    meet();
                    const float big = fmaxf(fmaxf(s_join[w][0][lane], s_join[w][1][lane]), fmaxf(s_join[w][2][lane], s_join[w][3][lane]));
                    const float was = -refs[lane];
                    const float now = big > was + kSlack ? big + kHead : was;
                    const float factor = exp2_of(was - now);  // 0 from before the first score
                    meet();
                    if (quarter == 0) refs[lane] = -now;
                    if (s > 0) {
                        wait(PV_DONE + (set ^ 1), ((k - 1) >> 1) & 1);
                        tmem_fence_after();
                        tmem_ld32(to, v);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float f0 = __shfl_sync(0xffffffffu, factor, 2 * i), f1 = __shfl_sync(0xffffffffu, factor, 2 * i + 1);
                        l[i] = mul_pair(l[i], pair_of(f0, f1));
                        v[2 * i] = __float_as_uint(__uint_as_float(v[2 * i]) * f0);
                        v[2 * i + 1] = __float_as_uint(__uint_as_float(v[2 * i + 1]) * f1);
                    }
                    if (s > 0) {
                        tmem_st32(to, v);
                        tmem_wait_st();
                        tmem_fence_before();
                    }
                    meet();
                    exponents();
                }
                // weights: into the sums, and as halves over the step's K
                uint8_t *weights = smem + C::kK + (k % kKStages) * C::kKBytes + slot * 128;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t z[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e0 = exp2_of(__uint_as_float(v[8 * u + 2 * i])), e1 = exp2_of(__uint_as_float(v[8 * u + 2 * i + 1]));
                        l[4 * u + i] = fma_pair(pair_of(e0, e1), ii, l[4 * u + i]);
                        z[i] = pack2<KVL_TYPE_HALF>(e0, e1);
                    }
                    *reinterpret_cast<uint4 *>(weights + (((4 * w + u) ^ (slot & 7)) << 4)) = make_uint4(z[0], z[1], z[2], z[3]);
                }
                fence_proxy_async_smem();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (P_FULL + set));
            }
            // ---- this share's part: rows' references and sums, then O
            const int rows = min(ROWS, job.s.e.fresh * G - job.tile * ROWS);
            const int part_number = job.before + job.job + int(blockIdx.x);
            float *part = a.prefix_parts + int64_t(part_number) * (ROWS * (D + 2));
            {
                float x[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 t = split_pair(l[i]);
                    x[2 * i] = t.x;
                    x[2 * i + 1] = t.y;
                }
                s_join[w][quarter][lane] = over_lanes(x, [](float y, float z) { return y + z; });
                meet();
                const int r = 32 * w + lane;
                if (quarter == 0 && r < rows && !*gone) {
                    part[r] = -refs[lane];
                    part[ROWS + r] = s_join[w][0][lane] + s_join[w][1][lane] + s_join[w][2][lane] + s_join[w][3][lane];
                }
                meet();
            }
            wait(PV_DONE + ((it + job.n - 1) & 1), ((it + job.n - 1) >> 1) & 1);
            tmem_fence_after();
            uint32_t v[32];
            tmem_ld32(lanes + 2 * ROWS, v);
            tmem_wait_ld();
            tmem_fence_before();
            if (slot < D && !*gone) {
                float *o = part + 2 * ROWS + 32 * w * D + slot;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (32 * w + i < rows) o[i * D] = __uint_as_float(v[i]);
            }
            if (tid == 0 && job.sa == 0 && !*gone) {
                const int64_t id = int64_t(job.s.e.row0) * G / ROWS + job.group + job.tile;
                const int from = int(cut.share_of(job.u0)), last = int(cut.share_of(job.u0 + job.s.steps - 1));
                reinterpret_cast<int2 *>(a.prefix_jobs)[id * H + job.h] = make_int2(part_number, last - from + 1);
            }
            it += job.n;
            ++jobs_done;
        } while (job.next(a));
    } else if (warp < kSoftmax + 4) {
        // ---- codes: groups 2 cw, 2 cw + 1 of every step
        const int cw = warp - kSoftmax;
        const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
        const int64_t v_plane_bytes = N * B * H * d;
        constexpr int kPer = 512 / D, kVecs = 2 * kGroup / kPer;  // rows of a warp's vector, vectors of its 32 slots
        // 8 lanes of a shared-memory phase write 4 chunks of an even and of an odd row: with the swizzle, 8
        // different 16-byte columns
        const int ch = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0), rw = D == 128 ? (lane >> 2) & 3 : lane >> 2;
        do {
            if (job.n == 0) continue;
            const int n = job.n, h = job.h, len = job.s.e.len, group = job.group;
            const int32_t *table = job.s.e.table;
            // Lane l looks after group l % 2 of the warp's two in step l / 2 of a batch of 16: its page, place and
            // scales.  The next batch's are fetched while this one is worked on.
            auto place = [&](int s, int &t0, int &nv) -> int32_t {
                t0 = nv = 0;
                const int g = (job.sa + s) * kGroups + cw * 2 + (lane & 1);
                if (s >= n) return -1;
                const int blk = g / per_block, at = (g - blk * per_block) * kGroup;
                t0 = blk * B + at;
                nv = min(min(kGroup, B - at), len - t0);
                if (nv <= 0) {
                    nv = 0;
                    return -1;
                }
                const int32_t page = table[blk];
                if (page < 0 || page >= N) {
                    report(a.report, KVL_ERANGE, a.shared.groups[group]);
                    nv = 0;
                    return -1;
                }
                return page;
            };
            auto scales = [&](int32_t page, float &ks, float &vs) {
                ks = 0.f;
                vs = 1.f;
                if (page >= 0) {
                    ks = __ldg(a.cache.scales + (plane + page) * H + h);
                    vs = v_scale(__ldg(a.cache.scales + (plane + N + page) * H + h));
                }
            };
            int t0, nv, t0n, nvn;
            int32_t page = place(lane >> 1, t0, nv), page_n = place(16 + (lane >> 1), t0n, nvn);
            float ks, vs, ksn = 0.f, vsn = 1.f;
            // Unit q, K (even) or V codes of step q / 2, comes by asynchronous copies, each vector to the thread that
            // takes it on from there.
            const uint8_t *src[2];
            int valid[2];
            uint32_t asked = 0;
            auto ask = [&](int base) {
                const uint32_t q = asked++;
                if (q < 2u * n) {
                    if ((q & 1) == 0) {
                        const int s = int(q >> 1);
                        const bool ahead = s - base >= 16;
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int from = ((s & 15) << 1) | y;
                            const int32_t pg = __shfl_sync(0xffffffffu, ahead ? page_n : page, from);
                            const int tt = __shfl_sync(0xffffffffu, ahead ? t0n : t0, from);
                            valid[y] = __shfl_sync(0xffffffffu, ahead ? nvn : nv, from);
                            if (ch * 16 >= d) valid[y] = 0;
                            src[y] = codes + (((plane + max(pg, 0)) * B + tt % B) * H + h) * d;
                        }
                    }
                    const uint32_t to = sm + C::kRing + (q % C::kUnits) * C::kUnitBytes + (tid - kSoftmax * 32) * 16;
                    const int64_t at = (q & 1) ? v_plane_bytes : 0;
#pragma unroll
                    for (int x = 0; x < kVecs; ++x) {
                        const int r = (x % (kVecs / 2)) * kPer + rw, y = x / (kVecs / 2);
                        const bool ok = r < valid[y];
                        copy_async16(to + x * 2048, src[y] + at + (ok ? int64_t(r) * H * d + ch * 16 : 0), ok);
                    }
                }
                copy_async_commit();
            };
            auto convert = [&](uint32_t q, uint8_t *dst) {
                const uint32_t from = sm + C::kRing + (q % C::kUnits) * C::kUnitBytes + (tid - kSoftmax * 32) * 16;
#pragma unroll
                for (int x = 0; x < kVecs; ++x) {
                    const uint4 z = ld_shared_v4(from + x * 2048);
                    const int r = cw * 2 * kGroup + x * kPer + rw;
                    uint4 lo, hi;
                    codes_of<CODE>(z.x, lo.x, lo.y);
                    codes_of<CODE>(z.y, lo.z, lo.w);
                    codes_of<CODE>(z.z, hi.x, hi.y);
                    codes_of<CODE>(z.w, hi.z, hi.w);
                    uint8_t *p = dst + (ch >> 2) * (kSlots * 128) + r * 128;
                    const int un = (ch & 3) * 2;
                    *reinterpret_cast<uint4 *>(p + ((un ^ (r & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4 *>(p + (((un + 1) ^ (r & 7)) << 4)) = hi;
                }
            };
#pragma unroll
            for (int x = 0; x < C::kUnits; ++x) ask(0);
            scales(page, ks, vs);
            {
                // ---- the job's rows, scaled by one power of two, which takes their largest element into [2^14, 2^15) (what
                // is lost is below 2^-39 of it), once the products of the job before are done
                const int rows = min(ROWS, job.s.e.fresh * G - job.tile * ROWS), set = jobs_done & 1;
                constexpr int kLanes = D / 8, kRowsPer = 32 / kLanes, kTurns = ROWS / (4 * kRowsPer);  // lanes of a row, rows of a warp's vector
                const int at = (lane % kLanes) * 8;
                uint4 raw[kTurns];
                float amax = 0.f;  // of finite elements
#pragma unroll
                for (int x = 0; x < kTurns; ++x) {
                    const int r = (cw + 4 * x) * kRowsPer + lane / kLanes;
                    raw[x] = make_uint4(0, 0, 0, 0);
                    if (r < rows && at < d) {
                        const uint32_t row = job.tile * ROWS + r, tok = row / uint32_t(G);
                        raw[x] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.attn.q.data) + (int64_t(job.s.e.row0) + tok) * a.attn.q.row_stride +
                                                                  int64_t(h * G + row - tok * G) * a.attn.q.head_stride + 2 * at);
                    }
                }
                auto floats = [&](const uint4 &x, float (&v)[8]) {
                    if (a.attn.type == KVL_TYPE_BFLOAT) load8<KVL_TYPE_BFLOAT>(reinterpret_cast<const uint8_t *>(&x), v);
                    else load8<KVL_TYPE_HALF>(reinterpret_cast<const uint8_t *>(&x), v);
                };
#pragma unroll
                for (int x = 0; x < kTurns; ++x) {
                    float v[8];
                    floats(raw[x], v);
#pragma unroll
                    for (int y = 0; y < 8; ++y) amax = fmaxf(amax, isfinite(v[y]) ? fabsf(v[y]) : 0.f);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                if (lane == 0) s_most[cw] = amax;
                asm volatile("bar.sync 3, 128;" ::: "memory");
                amax = fmaxf(fmaxf(s_most[0], s_most[1]), fmaxf(s_most[2], s_most[3]));
                // 2^e <= amax < 2^(e + 1), e held to what leaves both factors normal
                const int ex = max(-100, int(__float_as_uint(amax) >> 23) - 127);
                const float up = __uint_as_float(uint32_t(14 - ex + 127) << 23), down = __uint_as_float(uint32_t(ex - 14 + 127) << 23);
                if (it > 0) wait(K_EMPTY + (it - 1) % kKStages, ((it - 1) / kKStages) & 1);
#pragma unroll
                for (int x = 0; x < kTurns; ++x) {
                    const int r = (cw + 4 * x) * kRowsPer + lane / kLanes;
                    float v[8];
                    floats(raw[x], v);
                    uint4 z;
                    z.x = pack2<KVL_TYPE_HALF>(v[0] * up, v[1] * up);
                    z.y = pack2<KVL_TYPE_HALF>(v[2] * up, v[3] * up);
                    z.z = pack2<KVL_TYPE_HALF>(v[4] * up, v[5] * up);
                    z.w = pack2<KVL_TYPE_HALF>(v[6] * up, v[7] * up);
                    const int un = at / 8;
                    *reinterpret_cast<uint4 *>(smem + C::kQ + (un >> 3) * (ROWS * 128) + r * 128 + (((un & 7) ^ (r & 7)) << 4)) = z;
                    if (at == 0) s_refs[set][r] = -kNoScore;
                }
                if (cw == 0 && lane == 0) s_factor[set] = a.attn.sm_scale * kLog2e * down;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * Q_FULL);
                asm volatile("bar.sync 3, 128;" ::: "memory");  // (s_most is free again)
            }
            int base = 0;
            for (int s = 0; s < n; ++s) {
                if (s - base == 16) {
                    base += 16;
                    page = page_n; t0 = t0n; nv = nvn; ks = ksn; vs = vsn;
                    page_n = place(base + 16 + (lane >> 1), t0n, nvn);
                }
                if (s - base == 4) scales(page_n, ksn, vsn);
                const uint32_t k = it + s, kst = k % kKStages, vst = k % kVStages;
                wait(K_EMPTY + kst, ((k / kKStages) & 1) ^ 1);
                if (lane >> 1 == (s & 15)) {
                    Places &pl = places[k % kPlaces];
                    const int g = cw * 2 + (lane & 1);
                    pl.ks[g] = ks;
                    pl.lvs[g] = __log2f(vs);
                    pl.ivs[g] = __fdividef(1.f, vs);
                    pl.nv[g] = nv;
                }
                copy_async_wait<C::kUnits - 1>();
                convert(2 * s, smem + C::kK + kst * C::kKBytes);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (K_FULL + kst));
                ask(base);
                wait(V_EMPTY + vst, ((k / kVStages) & 1) ^ 1);
                copy_async_wait<C::kUnits - 1>();
                convert(2 * s + 1, smem + C::kV + vst * C::kVBytes);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (V_FULL + vst));
                ask(base);
            }
            it += n;
            ++jobs_done;
        } while (job.next(a));
    } else {
        // ---- products
        const uint32_t one = elect_one();
        auto scores = [&](uint32_t k) {  // S^T = K Q^T of step k
            wait(K_FULL + k % kKStages, (k / kKStages) & 1);
            tmem_fence_after();
            uint64_t kd = matrix_desc(sm + C::kK + (k % kKStages) * C::kKBytes, 16, 1024), qd = matrix_desc(sm + C::kQ, 16, 1024);
#pragma unroll 1
            for (int y = 0; y < D / 64; ++y) {
#pragma unroll
                for (int z = 0; z < 4; ++z) mma_smem(one, tmem + (k & 1) * ROWS, kd + 2 * z, qd + 2 * z, instr_desc(ROWS, false), y + z > 0);
                kd += kSlots * 128 >> 4;
                qd += ROWS * 128 >> 4;
            }
            mma_commit(one, bar + 8 * (S_FULL + (k & 1)));
            if (one) mbar_arrive(bar + 8 * (S_FULL + (k & 1)));
            __syncwarp();
        };
        do {
            if (job.n == 0) continue;
            wait(Q_FULL, jobs_done & 1);
            scores(it);
            for (int s = 0; s < job.n; ++s) {
                const uint32_t k = it + s;
                if (s + 1 < job.n) scores(k + 1);  // (its accumulators: the softmax has passed on the weights of k - 1)
                wait(V_FULL + k % kVStages, (k / kVStages) & 1);
                wait(P_FULL + (k & 1), (k >> 1) & 1);
                tmem_fence_after();
                uint64_t vd = matrix_desc(sm + C::kV + (k % kVStages) * C::kVBytes, kSlots * 128, 1024);
                uint64_t pd = matrix_desc(sm + C::kK + (k % kKStages) * C::kKBytes, kSlots * 128, 1024);
#pragma unroll
                for (int z = 0; z < kSlots / 16; ++z) {
                    mma_smem(one, tmem + 2 * ROWS, vd, pd, instr_desc(ROWS, true) | 1u << 15, s + z > 0);  // (A too is MN-major)
                    vd += 2048 >> 4;
                    pd += 2048 >> 4;
                }
                mma_commit(one, bar + 8 * (PV_DONE + (k & 1)));
                mma_commit(one, bar + 8 * (V_EMPTY + k % kVStages));
                mma_commit(one, bar + 8 * (K_EMPTY + k % kKStages));
            }
            it += job.n;
            ++jobs_done;
        } while (job.next(a));
        // the products in flight end (bounded) before their memory goes
        mma_commit(one, bar + 8 * LEAVE);
        mbar_wait_bounded(bar + 8 * LEAVE, 0);
    }
    __syncthreads();
    if (*gone && tid == 0) report(a.report, KVL_ETIMEOUT, blockIdx.x);
    if (warp == kWarps - 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int CODE, int D>
kvl_status launch_prefix(const AttendArgs &a, int sms, void *stream)
{
    static std::atomic<unsigned long long> ready[kMaxDevices];
    using C = Prefix<D>;
    if (!allow_smem(attend_prefix_kernel<CODE, D>, ready, C::kSmem)) return KVL_ECUDA;
    attend_prefix_kernel<CODE, D><<<sms, kThreads, C::kSmem, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}

template <int CODE>
kvl_status launch_prefix_dim(const AttendArgs &a, int sms, void *stream)
{
    return a.cache.head_dim <= 64 ? launch_prefix<CODE, 64>(a, sms, stream)
                                  : launch_prefix<CODE, 128>(a, sms, stream);
}

}  // namespace

kvl_status launch_attend_prefix(const AttendArgs &a, int sms, void *stream)
{
    return a.cache.code_type == KVL_CODE_FLOAT ? launch_prefix_dim<KVL_CODE_FLOAT>(a, sms, stream)
                                               : launch_prefix_dim<KVL_CODE_INT>(a, sms, stream);
}

}  // namespace kvl

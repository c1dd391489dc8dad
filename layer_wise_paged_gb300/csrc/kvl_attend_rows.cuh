// kvl_attend_rows.cuh -- attention of few rows a sequence: decoded tokens, drafted tokens.
//
// Each cached byte is read once, and 2 * 8 multiply-adds a byte are far below the tensor rate, so what counts
// is bytes in flight and few instructions a byte (256 ragged sequences: 242 us, 5.4 TB/s with 42 % of the
// issue slots used; one token of 128,000: 61 us, of which 8 pass before the first bytes have come).
//
// A warp takes 16 tokens of one KV head at a time from its own ring in shared memory (filled by
// 16-byte asynchronous copies, a pair of groups ahead, no barrier between warps) and computes the
// transposed products with 16 x 8 x 16 tensor instructions:
//   S^T [16 tokens x 8 rows] = K [16 x d] Q^T,   O^T [d x 8 rows] += V^T [d x 16] P^T.
// Tokens (then elements of V) fill the 16-high operand and the rows, i.e. the query heads of
// the KV head times the fresh tokens, the 8-wide one: a group of 4 or 8 heads wastes half or
// nothing where rows in the high operand would waste three quarters.  The order of elements
// in a product's inner dimension is free, so a lane reads its codes as 16-byte vectors, converts
// them in registers and needs no transposition; P^T comes out of S^T by an 8 x 8 register
// transpose.
//
// Work: every (entry, KV head, row tile) is a job of as many units as it has groups; the units
// of all jobs in a row are cut into equal contiguous shares, one a CTA, so a long sequence is
// split over many CTAs and short ones share one.  A job's groups are dealt to the CTA's warps,
// whose results are joined in shared memory; a job that crosses shares leaves its parts in the
// workspace and the CTA that finishes last joins them, in order of the shares.
//
// The kernel serves whole sequences, and the parts of attention over a shared prefix.
#pragma once

#include "kvl_attend.cuh"

namespace kvl {
namespace {

constexpr int kWarps = 6;
constexpr int kThreads = kWarps * 32;
constexpr int kPair = 2;          // groups a warp takes at a time (4 at d = 64: 137 us for 256 sequences of 1,500, with 2 123)
constexpr int kStages = 2;        // pairs in its ring: one worked on, one on its way (3 or 4 at d = 64: the same time)
constexpr int kCtasPerSm = 2;     // 12 warps an SM: 168 registers a thread, 192 KB of rings at d = 128 (3 at
                                  // d = 64: 142 us for those 123, as the registers run out)
// Units of a share: a job's groups, and kJobCost before them for starting and joining it (8 to 64 rows of
// 48 ragged sequences: 45 us, with a cost of 16 49; 256 sequences: 242 us and 249).  A share is at least
// kUnitsPerCta (8 heads of 1,500 tokens: 13 us, with 40 18), and a job of at most kSmallJob groups is not
// split, as its parts would have to be joined (one token of 777, 8 jobs of 49 groups: not split 15.9 us,
// split 13.5; of 500, 32 groups: 11.5 either way; with nothing kept whole and shares of 40 17.6).  The same
// values serve d = 64: 16 rows of 48 sequences of 3,000 (int8) 35.1 us, with a cost of 16 35.5, of 96 39.0;
// 256 sequences of 1,500 122.5 with any; one token of 1,500 10.5, with shares of 40 13.0, with jobs of up to
// 96 groups whole 14.6, with none whole 10.5.
constexpr int kJobCost = 48;
// (A job of the parts of a shared prefix costs less, as the join is another kernel's: 48 prompts of 18 rows on 2,200
// and their own tokens 62 us with 28, 66 with 22, 63 with 34, 67 with 48; 100 groups of 2 on 1,000 135, 138, 137, 139;
// 18 for own tokens and 40 for groups 72, 28 and 48 67.  CTAs of 4 warps, 3 an SM: 59.5, but 3 branches of 2,000
// 15.9 for 14.8.)
constexpr int kPartJobCost = 28;
constexpr int kUnitsPerCta = 12;
constexpr int kSmallJob = 48;

template <int D, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kGroupBytes = kGroup * D;            // K or V of a group
    static constexpr int kRing = kStages * kPair * 2 * kGroupBytes;  // one warp's ring
    static constexpr int kORow = D + 4;                       // floats; the pad spreads rows over banks
    static constexpr int kOBytes = kRows * kORow * 4;         // one warp's O, over its ring
    static constexpr int kWarpBytes = kRing > kOBytes ? kRing : kOBytes;
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kSmem = kQBytes + kWarps * kWarpBytes;
    static constexpr int kPartFloats = kRows * (D + 2);       // m, l, O of a part
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// The same of a V tile, whose rows 2(lane%4) and chunk(s) lane/4 a lane reads.
template <int D>
__device__ __forceinline__ uint32_t v_at(int r, int c)
{
    if constexpr (D == 64)
        return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (r & 6)) << 4);
    else if constexpr (D == 128)
        return r * 128 + ((c ^ (r & 6)) << 4);
    else
        return r * 256 + ((c ^ (((r >> 1) & 1) | (r & 4))) << 4);
}

// What a batch entry costs.  With PARTS the first n_seq are the sequences' own tokens, behind the ones they share, and
// those after them (with a.few) the groups' shared tokens.
template <int NT, bool PARTS>
__device__ __forceinline__ Cost cost_of(const AttendArgs &a, const HeldGroups *held, int i, void *rep)
{
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup;
    Cost c;
    c.lo = 0;
    if constexpr (PARTS) {
        if (i >= a.seqs.n_seq) {
            c.e = load_group(a, i - a.seqs.n_seq, rep);
        } else {
            c.e = load_entry(a.seqs, B, i, rep);
            const Sharing s = sharing_of(a, *held, c.e, i, rep);
            c.lo = max(s.tokens, 0);
            if (s.tokens < 0) c.e.len = c.e.fresh = 0;
        }
    } else {
        c.e = load_entry(a.seqs, B, i, rep);
        c.lo = first_seen(a, c.e.len - c.e.fresh);
    }
    const int64_t rows = int64_t(c.e.fresh) * (a.attn.n_heads / a.cache.n_kv_heads);
    c.tiles = rows > a.max_rows ? 0 : int32_t((rows + 8 * NT - 1) / (8 * NT));
    c.g0 = group_of(c.lo, B, per_block);
    // a sequence of no tokens is one group of none: its rows still get their zeros
    c.groups = max(1, c.e.len > 0 ? group_of(c.e.len - 1, B, per_block) + 1 - c.g0 : 0);
    return c;
}

template <int CODE, int TYPE, int D, int NT, bool PARTS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attend_rows_kernel(const __grid_constant__ AttendArgs a)
{
    using S = Shape<D, NT>;
    constexpr int kRows = S::kRows, kChunks = D / 16, kLaneBytes = D / 8, kCost = PARTS ? kPartJobCost : kJobCost;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_scan[kWarps];
    __shared__ uint32_t s_off, s_u[2];
    __shared__ Cost s_cost;
    __shared__ int s_entry, s_last;
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_cq[kRows];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nn = lane >> 2, kk = lane & 3;
    const int H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int G = a.attn.n_heads / H, per_block = (B + kGroup - 1) / kGroup;
    const int64_t N = a.cache.pool_blocks;

    const HeldGroups *held = nullptr;
    if constexpr (PARTS) {
        __shared__ HeldGroups s_groups;
        held = &s_groups;
        allow_dependents_launch();
        if (blockIdx.x == 0 && tid == 0) a.parts_done[2] = 0;
        const bool falls = hold_groups(a, s_groups);
        __syncthreads();
        // Of groups, or starts (below), that descend the rows of two may have one place among the parts.
        if (blockIdx.x == 0 && falls) a.parts_done[2] = 1;
        for (int i = int(blockIdx.x) * kThreads + int(threadIdx.x); i < a.seqs.n_seq; i += int(gridDim.x) * kThreads) {
            const Entry e = load_entry(a.seqs, a.cache.block_tokens, i, nullptr);
            Sharing s = sharing_of(a, s_groups, e, i, nullptr);
            if (!e.table) s.tokens = -1;
            reinterpret_cast<Sharing *>(a.sharing)[i] = s;
        }
    }
    // ---- this CTA's share of the units ----
    const int n_seq = a.seqs.n_seq + (PARTS && a.few ? a.shared.n_groups : 0), per_thread = (n_seq + kThreads - 1) / kThreads;
    const int i0 = min(n_seq, tid * per_thread), i1 = min(n_seq, i0 + per_thread);
    auto units_of = [&](const Cost &q) { return uint64_t(H * q.tiles) * uint32_t(q.groups + kCost); };
    Cost c;  // of the thread's last entry; kept where it is the only one
    uint64_t mine = 0;
    for (int i = i0; i < i1; ++i) {
        c = cost_of<NT, PARTS>(a, held, i, blockIdx.x == 0 ? a.report : nullptr);
        mine += units_of(c);
        if constexpr (PARTS)
            if (blockIdx.x == 0 && i < a.seqs.n_seq && a.seqs.starts[i + 1] < a.seqs.starts[i]) a.parts_done[2] = 1;
    }
    uint64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    uint64_t before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    if constexpr (PARTS)
        if (blockIdx.x == 0 && tid == 0) a.parts_done[0] = total < kMostUnits;
    if (total == 0 || total >= kMostUnits) {
        if (total && blockIdx.x == 0 && tid == 0) report(a.report, KVL_ERANGE, n_seq);
        return;
    }
    const Cut cut(uint32_t(total), min(gridDim.x, (uint32_t(total) + kUnitsPerCta - 1) / kUnitsPerCta));
    if (blockIdx.x >= cut.shares) return;
    // The share's first unit and the next share's: where one falls inside a small job it moves to the
    // job's start.
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const uint64_t x = cut.start(blockIdx.x + k);
        if (x >= before && x < before + mine) {
            uint64_t at = before;
            int i = i0;
            if (per_thread > 1)
                for (;; ++i) {
                    c = cost_of<NT, PARTS>(a, held, i, nullptr);
                    if (x < at + units_of(c)) break;
                    at += units_of(c);
                }
            uint32_t in = uint32_t(x - at);
            if (c.groups <= kSmallJob) in -= in % (c.groups + kCost);
            if (k == 0) {
                s_entry = i;
                s_off = in;
                s_cost = c;
            }
            s_u[k] = uint32_t(at) + in;
        } else if (tid == 0 && x == total) {
            s_u[k] = uint32_t(total);
        }
    }
    __syncthreads();
    uint32_t u = s_u[0];
    const uint32_t u_end = s_u[1];
    int entry = s_entry;
    uint32_t off = s_off;  // units of the entry before u
    c = s_cost;

    const uint32_t ring = smem_u32(smem) + S::kQBytes + warp * S::kWarpBytes;
    __half *sq = reinterpret_cast<__half *>(smem);
    const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
    const int64_t plane = int64_t(a.layer) * 2 * N, v_plane_bytes = N * B * H * d;

    while (u < u_end) {
        while (off >= units_of(c)) {  // on to the entry that holds unit u
            off -= uint32_t(units_of(c));
            c = cost_of<NT, PARTS>(a, held, ++entry, nullptr);
        }
        const uint32_t per_job = c.groups + kCost;
        const int job = int(off / per_job), in = int(off - job * per_job);
        const int taken = int(min(per_job - in, u_end - u));
        const int ga = max(0, in - kCost), gb = max(0, in + taken - kCost);
        const uint32_t group0 = u - in + kCost;  // the unit of the job's first group
        off += taken;
        u += taken;
        if (ga == gb) continue;  // its groups are the next share's
        const int h = job / c.tiles, tile = job - h * c.tiles;
        const int rows = min(kRows, c.e.fresh * G - tile * kRows);
        const int pos0 = c.e.len - c.e.fresh;
        const bool of_group = PARTS && entry >= a.seqs.n_seq;  // the shared tokens of a group

        // ---- groups of this warp: pair k holds ga + 2 (warp + kWarps k) and the next.  Lane l looks after
        // group l % 2 of pair l / 2 of a batch of 16: its page, scales and place; the next batch's are
        // fetched while this one is worked on.
        const int count = (gb - ga - kPair * warp + kPair * kWarps - 1) / (kPair * kWarps);  // may be <= 0
        auto place_of = [&](int k, int &t0, int &nv) -> int32_t {  // page of this lane's group of pair k, -1: none
            t0 = 0;
            nv = 0;
            const int g = ga + kPair * (warp + kWarps * k) + (lane & 1);
            if (g >= gb) return -1;
            const int blk = (c.g0 + g) / per_block, slot = (c.g0 + g - blk * per_block) * kGroup;
            t0 = blk * B + slot;
            nv = min(min(kGroup, B - slot), c.e.len - t0);
            if (nv <= 0) return -1;
            const int32_t page = c.e.table[blk];
            if (page < 0 || page >= N) {
                report(a.report, KVL_ERANGE, of_group ? a.shared.groups[entry - a.seqs.n_seq] : entry);
                nv = 0;
                return -1;
            }
            return page;
        };
        auto scales_of = [&](int32_t page, float &ks, float &lvs, float &ivs) {
            ks = 1.f;
            float vs = 1.f;
            if (page >= 0) {
                ks = __ldg(a.cache.scales + (plane + page) * H + h);
                vs = v_scale(__ldg(a.cache.scales + (plane + N + page) * H + h));
            }
            lvs = __log2f(vs);
            ivs = __fdividef(1.f, vs);
        };
        int t0_l, nv_l, t0_n, nv_n;
        int32_t page_l = place_of(lane >> 1, t0_l, nv_l), page_n = -1;
        float ks_l, lvs_l, ivs_l, ks_n = 1.f, lvs_n = 0.f, ivs_n = 1.f;

        // start of pair k's copies (its pages are of this batch or the next)
        int base_k = 0;
        const int row_l = lane / kChunks, ch_l = lane % kChunks;  // this lane's row and 16 bytes of a 512-byte instruction
        const int row_bytes = H * d;
        auto load_pair = [&](int k) {
            if (k < count) {
                const bool ahead = k - base_k >= 16;
                const uint32_t dst = ring + (k % kStages) * (kPair * 2 * S::kGroupBytes);
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    const int from = ((k & 15) << 1) | y;
                    const int32_t page = __shfl_sync(0xffffffffu, ahead ? page_n : page_l, from);
                    const int t0 = __shfl_sync(0xffffffffu, ahead ? t0_n : t0_l, from);
                    const int nv = __shfl_sync(0xffffffffu, ahead ? nv_n : nv_l, from);
                    const uint8_t *src = codes + (((plane + max(page, 0)) * B + t0 % B) * H + h) * d;
                    const uint32_t dk = dst + y * (2 * S::kGroupBytes);
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        const int r = x * (32 / kChunks) + row_l;
                        const bool ok = r < nv && ch_l * 16 < d;  // (past the head lies the next one, or the end of the pool)
                        const uint8_t *p = src + (ok ? r * row_bytes + ch_l * 16 : 0);
                        copy_async16(dk + k_at<D>(r, ch_l), p, ok);
                        copy_async16(dk + S::kGroupBytes + v_at<D>(r, ch_l), p + v_plane_bytes, ok);
                    }
                }
            }
            copy_async_commit();
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) load_pair(k);

        // ---- Q: each row scaled by a power of two into the range of a half (undone in s_cq), which is exact
        // but for elements below 2^-14 of the row's largest (2^-25 of it at most).  A warp's rows are all on
        // their way before the first is looked at.
        constexpr int kQTurns = (kRows + kWarps - 1) / kWarps;
        uint32_t qraw[kQTurns][D / 64];
#pragma unroll
        for (int z = 0; z < kQTurns; ++z) {
            const int r = warp + z * kWarps, row = tile * kRows + r;
            const bool ok = r < rows;
            const uint8_t *src = static_cast<const uint8_t *>(a.attn.q.data) +
                                 (int64_t(c.e.row0) + (ok ? row / G : 0)) * a.attn.q.row_stride +
                                 int64_t(h * G + (ok ? row % G : 0)) * a.attn.q.head_stride;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const int e = lane * 2 + 64 * x;
                qraw[z][x] = ok && e < d ? *reinterpret_cast<const uint32_t *>(src + 2 * e) : 0;
            }
        }
#pragma unroll
        for (int z = 0; z < kQTurns; ++z) {
            const int r = warp + z * kWarps;
            float v[D / 32];
            float amax = 0.f;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const uint32_t w = qraw[z][x];
                if constexpr (TYPE == KVL_TYPE_BFLOAT) {
                    v[2 * x] = __uint_as_float(w << 16);
                    v[2 * x + 1] = __uint_as_float(w & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                    v[2 * x] = f.x;
                    v[2 * x + 1] = f.y;
                }
                amax = fmaxf(amax, fmaxf(fabsf(v[2 * x]), fabsf(v[2 * x + 1])));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (r >= kRows) break;
            // amax * up in [1, 2) (exact powers of two; a row of zeros or infinities stays)
            const uint32_t ex = (__float_as_uint(amax) >> 23) & 0xffu;
            const bool plain = ex < 2 || ex > 252;
            const float up = plain ? 1.f : __uint_as_float((254u - ex) << 23);
            const float down = plain ? 1.f : __uint_as_float(ex << 23);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
                *reinterpret_cast<__half2 *>(sq + r * D + lane * 2 + 64 * x) =
                    __floats2half2_rn(v[2 * x] * up, v[2 * x + 1] * up);
            if (lane == 0) s_cq[r] = a.attn.sm_scale * kLog2e * down;
        }
        scales_of(page_l, ks_l, lvs_l, ivs_l);
        page_n = place_of(16 + (lane >> 1), t0_n, nv_n);
        __syncthreads();

        // visible tokens of this lane's columns (rows 2kk, 2kk + 1 of each tile of 8) and of all rows
        int lo[NT][2], hi[NT][2];
        float cq[NT][2];
        const int first_pos = pos0 + (tile * kRows) / G, last_pos = pos0 + (tile * kRows + rows - 1) / G;
        const bool causal = !of_group && a.attn.causal;
        auto first_token = [&](int pos) { return PARTS ? c.lo : first_seen(a, pos); };
        const int all_hi = causal ? min(c.e.len, first_pos + 1) : c.e.len;
        const int all_lo = first_token(last_pos);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = 8 * t + 2 * kk + x;
                const int pos = pos0 + (tile * kRows + r) / G;
                hi[t][x] = causal ? min(c.e.len, pos + 1) : c.e.len;
                lo[t][x] = first_token(pos);
                if (r >= rows) { lo[t][x] = 0; hi[t][x] = c.e.len; }
                cq[t][x] = s_cq[r];
            }

        float o[NT][kChunks][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int x = 0; x < kChunks; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
        }

        for (int k = 0; k < count; ++k) {
            if (k - base_k == 16) {
                base_k += 16;
                page_l = page_n; t0_l = t0_n; nv_l = nv_n; ks_l = ks_n; lvs_l = lvs_n; ivs_l = ivs_n;
                page_n = place_of(base_k + 16 + (lane >> 1), t0_n, nv_n);
            }
            if (k - base_k == 6) scales_of(page_n, ks_n, lvs_n, ivs_n);
            load_pair(k + kStages - 1);
            copy_async_wait<kStages - 1>();
            __syncwarp();
            float ks[kPair], lvs[kPair], ivs[kPair];
            int t0[kPair], nv[kPair];
            bool whole = true;
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                const int from = ((k & 15) << 1) | y;
                t0[y] = __shfl_sync(0xffffffffu, t0_l, from);
                nv[y] = __shfl_sync(0xffffffffu, nv_l, from);
                ks[y] = __shfl_sync(0xffffffffu, ks_l, from);
                lvs[y] = __shfl_sync(0xffffffffu, lvs_l, from);
                ivs[y] = __shfl_sync(0xffffffffu, ivs_l, from);
                whole = whole && nv[y] == kGroup && t0[y] >= all_lo && t0[y] + kGroup <= all_hi;
            }
            const uint8_t *kt = smem + (ring - smem_u32(smem)) + (k % kStages) * (kPair * 2 * S::kGroupBytes);

            // ---- S^T = K Q^T
            float s[NT][kPair][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int y = 0; y < kPair; ++y) s[t][y][0] = s[t][y][1] = s[t][y][2] = s[t][y][3] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const int ch = kk + 4 * i;
                uint32_t q[NT][8];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 *p = reinterpret_cast<const uint4 *>(sq + (8 * t + nn) * D + ch * 16);
                    const uint4 x = p[0], y = p[1];
                    q[t][0] = x.x; q[t][1] = x.y; q[t][2] = x.z; q[t][3] = x.w;
                    q[t][4] = y.x; q[t][5] = y.y; q[t][6] = y.z; q[t][7] = y.w;
                }
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    const uint8_t *kg = kt + y * (2 * S::kGroupBytes);
                    const uint4 ka = *reinterpret_cast<const uint4 *>(kg + k_at<D>(nn, ch));
                    const uint4 kb = *reinterpret_cast<const uint4 *>(kg + k_at<D>(nn + 8, ch));
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t a0, a1, a2, a3;
                        codes_of<CODE>(wa[w], a0, a2);
                        codes_of<CODE>(wb[w], a1, a3);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816(s[t][y], a0, a1, a2, a3, q[t][2 * w], q[t][2 * w + 1]);
                    }
                }
            }

            // ---- softmax over tokens nn, nn + 8 of each group, of columns 2kk, 2kk + 1.  Only a score that
            // has outgrown its column's reference makes the lanes compare theirs.
            bool grew = false;
            float top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[t][y][x] = fmaf(s[t][y][x], ks[y] * cq[t][x & 1], lvs[y]);
                        if (!whole) {
                            const int r = nn + 8 * (x >> 1);
                            if (r >= nv[y] || t0[y] + r < lo[t][x & 1] || t0[y] + r >= hi[t][x & 1]) s[t][y][x] = -INFINITY;
                        }
                        top[t][x & 1] = fmaxf(top[t][x & 1], s[t][y][x]);
                    }
                }
                grew = grew || top[t][0] > m[t][0] + kSlack || top[t][1] > m[t][1] + kSlack;
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v = top[t][x];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        if (v <= m[t][x] + kSlack || v == -INFINITY) continue;
                        const float f = exp2_of(m[t][x] - (v + kHead));
                        m[t][x] = v + kHead;
                        l[t][x] *= f;
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            o[t][j][x] *= f;
                            o[t][j][x + 2] *= f;
                        }
                    }
            }
            uint32_t p0[NT][kPair], p1[NT][kPair];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    float w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float ref = m[t][x & 1] == -INFINITY ? 0.f : m[t][x & 1];
                        w[x] = exp2_of(s[t][y][x] - ref);
                        if (whole || s[t][y][x] != -INFINITY) l[t][x & 1] = fmaf(w[x], ivs[y], l[t][x & 1]);
                    }
                    p0[t][y] = transpose8x8(pack2<KVL_TYPE_HALF>(w[0], w[1]));
                    p1[t][y] = transpose8x8(pack2<KVL_TYPE_HALF>(w[2], w[3]));
                }

            // ---- O^T += V^T P^T: tokens 2kk, 2kk + 1, 2kk + 8, 2kk + 9, elements from nn * D/8 on
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                const uint8_t *vt = kt + y * (2 * S::kGroupBytes) + S::kGroupBytes;
                uint32_t vw[4][kLaneBytes / 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 2 * kk + (r & 1) + 8 * (r >> 1);
                    if constexpr (D == 64) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(vt + v_at<D>(row, nn >> 1) + 8 * (nn & 1));
                        vw[r][0] = x.x; vw[r][1] = x.y;
                    } else {
#pragma unroll
                        for (int z = 0; z < D / 128; ++z) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(vt + v_at<D>(row, nn * (D / 128) + z));
                            vw[r][4 * z] = x.x; vw[r][4 * z + 1] = x.y; vw[r][4 * z + 2] = x.z; vw[r][4 * z + 3] = x.w;
                        }
                    }
                }
                // a NaN in a token that some rows do not see must not reach them through 0 * NaN
                bool has_nan = false;
                if (CODE == KVL_CODE_FLOAT && !whole) {
                    uint32_t nan_words = 0;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int x = 0; x < kLaneBytes / 4; ++x) nan_words |= __vcmpeq4(vw[r][x] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    has_nan = __any_sync(0xffffffffu, nan_words != 0);
                }
                if (has_nan) {
                    // NaN codes leave the product; a product of NaN marks with the rows' view of the tokens
                    // tells which results they belong to
#pragma unroll
                    for (int x = 0; x < kLaneBytes / 4; ++x) {
                        uint32_t w[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t bad = __vcmpeq4(vw[r][x] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            w[r] = bad & 0x38383838u;  // marks: the code of 1
                            vw[r][x] &= ~bad;
                        }
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t n0, n1, n2, n3;
                            codes_of<CODE>(__byte_perm(w[0], w[1], z ? 0x7362 : 0x5140), n0, n1);
                            codes_of<CODE>(__byte_perm(w[2], w[3], z ? 0x7362 : 0x5140), n2, n3);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                uint32_t see[2];
#pragma unroll
                                for (int u2 = 0; u2 < 2; ++u2)
                                    see[u2] = transpose8x8((s[t][y][2 * u2] != -INFINITY ? 0x3c00u : 0u) |
                                                           (s[t][y][2 * u2 + 1] != -INFINITY ? 0x3c000000u : 0u));
                                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816(hit, n0, n1, n2, n3, see[0], see[1]);
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (hit[q] > 0.f) o[t][2 * x + z][q] = NAN;
                            }
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < kLaneBytes / 4; ++x)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {  // elements 4x + 2z, 4x + 2z + 1 of the lane's run
                        uint32_t a0, a1, a2, a3;
                        codes_of<CODE>(__byte_perm(vw[0][x], vw[1][x], z ? 0x7362 : 0x5140), a0, a1);
                        codes_of<CODE>(__byte_perm(vw[2][x], vw[3][x], z ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16816(o[t][2 * x + z], a0, a1, a2, a3, p0[t][y], p1[t][y]);
                    }
            }
            __syncwarp();  // the stage may be filled again
        }
        copy_async_wait<0>();
        __syncwarp();

        // ---- join the warps
        float *so = reinterpret_cast<float *>(smem + S::kQBytes + warp * S::kWarpBytes);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = l[t][x];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int r = 8 * t + 2 * kk + x;
                if (nn == 0) {
                    s_m[warp][r] = m[t][x];
                    s_l[warp][r] = v;
                }
                if (r < rows) {
#pragma unroll
                    for (int y = 0; y < kLaneBytes / 4; ++y)
                        *reinterpret_cast<float4 *>(so + r * S::kORow + nn * kLaneBytes + 4 * y) =
                            make_float4(o[t][2 * y][x], o[t][2 * y][x + 2], o[t][2 * y + 1][x], o[t][2 * y + 1][x + 2]);
                }
            }
        }
        __syncthreads();
        const bool complete = ga == 0 && gb == c.groups;
        auto finish = [&](int r, int e, float4 v, float big, float sum) {  // 4 elements of a row's result
            if (e >= d) return;
            const int row = tile * kRows + r;
            const int64_t t = int64_t(c.e.row0) + row / G;
            const int head = h * G + row % G;
            if constexpr (PARTS) {
                const int64_t at = (t + (of_group ? a.seqs.n_rows : 0)) * a.attn.n_heads + head;
                *reinterpret_cast<float4 *>(a.row_o + at * D + e) = v;
                if (e == 0) *reinterpret_cast<float2 *>(a.row_ml + at * 2) = make_float2(big, sum);
                return;
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // 0: the row sees nothing
            uint8_t *dst = static_cast<uint8_t *>(a.attn.out.data) + t * a.attn.out.row_stride +
                           int64_t(head) * a.attn.out.head_stride + 2 * e;
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<TYPE>(v.x * inv, v.y * inv), pack2<TYPE>(v.z * inv, v.w * inv));
            if (e == 0 && a.attn.lse)
                a.attn.lse[t * a.attn.n_heads + head] = sum == 0.f ? -INFINITY : (big + __log2f(sum)) * (1.f / kLog2e);
        };
        float *part = a.parts + (int64_t(blockIdx.x) * 2 + (ga == 0 ? 1 : 0)) * S::kPartFloats;
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), e = (x % (D / 4)) * 4;
            float big = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) big = fmaxf(big, s_m[w][r]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = s_m[w][r] == -INFINITY ? 0.f : exp2_of(s_m[w][r] - big);
                const float4 y = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem + S::kQBytes + w * S::kWarpBytes) + r * S::kORow + e);
                v.x += y.x * f; v.y += y.y * f; v.z += y.z * f; v.w += y.w * f;
                sum += s_l[w][r] * f;
            }
            if (complete) {
                finish(r, e, v, big, sum);
            } else {
                *reinterpret_cast<float4 *>(part + 2 * kRows + r * D + e) = v;
                if (e == 0) {
                    part[r] = big;
                    part[kRows + r] = sum;
                }
            }
        }
        if (!complete) {
            // parts of this job: shares first .. last; the one that arrives last joins them
            const int first = int(cut.share_of(group0)), last = int(cut.share_of(group0 + c.groups - 1));
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(&a.counters[first], 1u) == uint32_t(last - first);
            __syncthreads();
            if (s_last) {
                __threadfence();
                if (tid == 0) a.counters[first] = 0;
                // The parts' maxima and sums into shared memory (over the rings), all loads at once; a warp a
                // row turns them into factors; then each warp adds up every kWarps-th part and the warps'
                // sums are added up in order (one token of 128,000, 38 parts of 8 rows: 62.4 us; with a thread an
                // element 64.9).
                const int n_parts = last - first + 1;
                float *fac = reinterpret_cast<float *>(smem + S::kQBytes), *sums = fac + n_parts * kRows;
                auto part_of = [&](int b) { return a.parts + (int64_t(first + b) * 2 + (b == 0)) * S::kPartFloats; };
                for (int x = tid; x < n_parts * kRows; x += kThreads) {
                    const int b = x / kRows, r = x % kRows;
                    fac[x] = r < rows ? __ldcg(part_of(b) + r) : 0.f;
                    sums[x] = r < rows ? __ldcg(part_of(b) + kRows + r) : 0.f;
                }
                __syncthreads();
                for (int r = warp; r < rows; r += kWarps) {
                    float big = -INFINITY, sum = 0.f;
                    for (int b = lane; b < n_parts; b += 32) big = fmaxf(big, fac[b * kRows + r]);
#pragma unroll
                    for (int x = 16; x; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
                    for (int b = lane; b < n_parts; b += 32) {
                        const float mb = fac[b * kRows + r], f = mb == -INFINITY ? 0.f : exp2_of(mb - big);
                        fac[b * kRows + r] = f;
                        sum += sums[b * kRows + r] * f;
                    }
#pragma unroll
                    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                    if (lane == 0) {
                        s_m[0][r] = big;
                        s_l[0][r] = sum;
                    }
                }
                __syncthreads();
                constexpr int kVecs = kRows * (D / 4) / 32;  // vectors of a lane
                float4 v[kVecs];
#pragma unroll
                for (int x = 0; x < kVecs; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int b = warp; b < n_parts; b += kWarps) {
                    const float *p = part_of(b) + 2 * kRows;
#pragma unroll
                    for (int x = 0; x < kVecs; ++x) {
                        const int r = (x * 32 + lane) / (D / 4);
                        if (r >= rows) continue;
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(p) + x * 32 + lane);
                        const float f = fac[b * kRows + r];
                        v[x].x += y.x * f; v[x].y += y.y * f; v[x].z += y.z * f; v[x].w += y.w * f;
                    }
                }
                __syncthreads();
                float4 *all = reinterpret_cast<float4 *>(smem + S::kQBytes);  // over the factors
#pragma unroll
                for (int x = 0; x < kVecs; ++x) all[(warp * kVecs + x) * 32 + lane] = v[x];
                __syncthreads();
                for (int x = tid; x < rows * (D / 4); x += kThreads) {
                    const int r = x / (D / 4), e = (x % (D / 4)) * 4;
                    float4 y = all[x];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) {
                        const float4 z = all[w * kVecs * 32 + x];
                        y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
                    }
                    finish(r, e, y, s_m[0][r], s_l[0][r]);
                }
            }
        }
        __syncthreads();  // Q, the rings and the joined results are free again
    }
}

template <int CODE, int TYPE, int D, int NT, bool PARTS>
kvl_status launch_rows(const AttendArgs &a, int sms, void *stream)
{
    static std::atomic<unsigned long long> ready[kMaxDevices];
    if (!allow_smem(attend_rows_kernel<CODE, TYPE, D, NT, PARTS>, ready, Shape<D, NT>::kSmem)) return KVL_ECUDA;
    // (rings of 256 elements leave room for one CTA an SM)
    const int ctas = sms * (2 * Shape<D, NT>::kSmem <= 220 * 1024 ? kCtasPerSm : 1);
    attend_rows_kernel<CODE, TYPE, D, NT, PARTS><<<ctas, kThreads, Shape<D, NT>::kSmem, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}

// Row tiles of 8 or 16 by the bound on an entry's rows: a tile's tokens are read and converted once.
// 16 rows of 256 elements would not leave a warp its registers.
template <int CODE, int TYPE, bool PARTS>
kvl_status launch_rows_dim(const AttendArgs &a, int64_t most, int sms, void *stream)
{
    // Row tiles of 8 while they hold all rows, else of 16, so that the cache is read half as often (256 sequences
    // of 1,500, 4 rows, d = 128: in tiles of 8 154 us, of 16 215; 40 of 3,000, 8 rows: 57 and 75).
    if (a.cache.head_dim <= 64) {
        if (most <= 8) return launch_rows<CODE, TYPE, 64, 1, PARTS>(a, sms, stream);
        return launch_rows<CODE, TYPE, 64, 2, PARTS>(a, sms, stream);
    }
    if (a.cache.head_dim <= 128)
        return most <= 8 ? launch_rows<CODE, TYPE, 128, 1, PARTS>(a, sms, stream) : launch_rows<CODE, TYPE, 128, 2, PARTS>(a, sms, stream);
    return launch_rows<CODE, TYPE, 256, 1, PARTS>(a, sms, stream);
}

template <bool PARTS>
kvl_status launch_rows_part(const AttendArgs &a, int64_t most, int sms, void *stream)
{
    const bool bf = a.attn.type == KVL_TYPE_BFLOAT;
    if (a.cache.code_type == KVL_CODE_FLOAT)
        return bf ? launch_rows_dim<KVL_CODE_FLOAT, KVL_TYPE_BFLOAT, PARTS>(a, most, sms, stream)
                  : launch_rows_dim<KVL_CODE_FLOAT, KVL_TYPE_HALF, PARTS>(a, most, sms, stream);
    return bf ? launch_rows_dim<KVL_CODE_INT, KVL_TYPE_BFLOAT, PARTS>(a, most, sms, stream)
              : launch_rows_dim<KVL_CODE_INT, KVL_TYPE_HALF, PARTS>(a, most, sms, stream);
}

}  // namespace
}  // namespace kvl

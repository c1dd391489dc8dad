// kvl_attend_chunk.cu -- attention of many rows a sequence: prompts and their chunks.
//
// Bound by the tensor cores: 4 d operations for each (row, visible token).  One CTA an SM takes
// 256 rows of one KV head (query heads of the head times tokens), two accumulator tiles of 128,
// and walks the tokens 128 slots (8 groups) at a time:
//   warps 0-3, 4-7   softmax of tile 0, tile 1: a thread a row.  S comes from tensor memory, P goes
//                    back over it as halves, O is rescaled in place when the maximum has grown
//                    by more than 2^8 since it was last set (rare after the first slots);
//   warps 8-11       read K and V codes from the pages, convert them to halves (exact) and lay
//                    them out in shared memory for the tensor cores (128-byte swizzle), two
//                    stages each, with the groups' scales and places beside them;
//   warp 12          one thread issues the products: S_g = Q_g K^T (both in shared memory, K-major)
//                    and O_g += P_g V (P in tensor memory, V token-major), for g = 0, 1 in turn,
//                    so one tile's softmax runs under the other tile's products.
// A converted K or V stage serves 256 rows, which is what keeps the conversion (16 bytes in, 32
// out a vector) small beside the products.
//
// Every wait on a barrier is bounded: past the limit a flag is raised, the report says
// KVL_ETIMEOUT, every role leaves, and the tensor memory is given back.
#include "kvl_attend.cuh"

namespace kvl {
namespace {

constexpr int kThreads = 512;
constexpr int kTileRows = 128;
constexpr int kJobRows = 2 * kTileRows;
constexpr int kSlots = 128;                 // slots of a step
constexpr int kGroups = kSlots / kGroup;    // 8
constexpr int kStages = 2;
constexpr int kPlaces = 4;                  // steps whose scales are kept (see place_full)
constexpr int kStepsPerCta = 2;             // a share is at least this many steps
constexpr float kSlack = 8.f;               // log2 of the largest weight before O is rescaled

// Scales and places of a step's groups; partial[w]: some row sees only a part of the two groups that
// converting warp w filled.
struct Places {
    float ks[kGroups], lvs[kGroups], ivs[kGroups];
    int32_t t0[kGroups], nv[kGroups];
    int32_t partial[4];
};

template <int D>
struct Chunk {
    static constexpr int kTileBytes = kTileRows * D * 2;  // Q tile, K or V stage: 128 rows of D halves
    static constexpr int kQ = 0;
    static constexpr int kK = 2 * kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    static constexpr int kSmem = kV + kStages * kTileBytes + 1024;  // and room to start on 1024
    static constexpr int kPartFloats = kJobRows * (D + 2);
};

// Barriers (each in its own 8 bytes).
enum Bar { K_FULL = 0, K_EMPTY = 2, V_FULL = 4, V_EMPTY = 6, S_FULL = 8, P_FULL = 10, PV_DONE = 12, BARS = 14 };

// ---- tensor-core wrappers -------------------------------------------------------------------

// Shared-memory matrix descriptor: 128-byte swizzle, addresses in 16-byte units.  K-major (rows of
// 64 halves): `stride` between groups of 8 rows.  MN-major: `lead` between runs of 64 elements
// of the non-contracted index, `stride` between groups of 8 contracted ones.
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t lead, uint32_t stride)
{
    return uint64_t((addr >> 4) & 0x3fff) | (uint64_t(lead >> 4) << 16) | (uint64_t(stride >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Instruction descriptor: f32 accumulators, half operands, 128 x n; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_mn)
{
    return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(kTileRows >> 4) << 24);
}

__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
}

__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}

__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
        : "memory");
}

// Bounded wait that also leaves when another role has given up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *gone)
{
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*gone) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *gone = 1;
            return false;
        }
    }
    return true;
}

// ---- work ------------------------------------------------------------------------------------

// Row tile `tile` of an entry: the tokens any of its rows sees, as steps of 128 slots.
struct Tile {
    int32_t rows;      // rows of this tile (at most kJobRows)
    int32_t g0, g1;    // groups
    int32_t steps;     // at least 1
    int32_t all_lo, all_hi;  // tokens every row sees
};

__device__ __forceinline__ Tile tile_of(const AttendArgs &a, const Entry &e, int tile)
{
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup, G = a.attn.n_heads / a.cache.n_kv_heads;
    Tile t;
    t.rows = int32_t(min(int64_t(kJobRows), int64_t(e.fresh) * G - int64_t(tile) * kJobRows));
    const int pos0 = e.len - e.fresh;
    const int first = pos0 + int(int64_t(tile) * kJobRows / G), last = pos0 + int((int64_t(tile) * kJobRows + t.rows - 1) / G);
    const int hi = a.attn.causal ? min(e.len, last + 1) : e.len;
    const int lo = a.attn.window > 0 ? max(0, first - a.attn.window + 1) : 0;
    t.all_hi = a.attn.causal ? min(e.len, first + 1) : e.len;
    t.all_lo = a.attn.window > 0 ? max(0, last - a.attn.window + 1) : 0;
    t.g0 = t.g1 = 0;
    if (hi > lo) {
        t.g0 = group_of(lo, B, per_block);
        t.g1 = group_of(hi - 1, B, per_block) + 1;
    }
    t.steps = max(1, (t.g1 - t.g0 + kGroups - 1) / kGroups);
    return t;
}

struct Share {
    Entry e;
    int32_t tiles;
    int64_t steps;  // of one KV head, all tiles
};

__device__ __forceinline__ Share share_of(const AttendArgs &a, int i, void *rep)
{
    Share s;
    s.e = load_entry(a.seqs, a.cache.block_tokens, i, rep);
    const int64_t rows = int64_t(s.e.fresh) * (a.attn.n_heads / a.cache.n_kv_heads);
    s.tiles = rows > a.max_rows ? int32_t((rows + kJobRows - 1) / kJobRows) : 0;
    s.steps = 0;
    for (int t = 0; t < s.tiles; ++t) s.steps += tile_of(a, s.e, t).steps;
    return s;
}

template <int CODE, int TYPE, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_chunk_kernel(const __grid_constant__ AttendArgs a)
{
    using C = Chunk<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long bars[BARS];
    __shared__ Places places[kPlaces];
    __shared__ float s_cq[kJobRows];
    __shared__ int64_t s_scan[kThreads / 32], s_off;
    __shared__ int s_entry, s_last, s_gone, s_nan;
    __shared__ uint32_t s_tmem;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int G = a.attn.n_heads / H, per_block = (B + kGroup - 1) / kGroup;
    const int64_t N = a.cache.pool_blocks;

    // ---- this CTA's share of the steps
    const int n_seq = a.seqs.n_seq, per_thread = (n_seq + kThreads - 1) / kThreads;
    const int i0 = min(n_seq, tid * per_thread), i1 = min(n_seq, i0 + per_thread);
    int64_t mine = 0;
    for (int i = i0; i < i1; ++i) mine += H * share_of(a, i, blockIdx.x == 0 ? a.report : nullptr).steps;
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    int64_t before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const int64_t shares = min(int64_t(gridDim.x), (total + kStepsPerCta - 1) / kStepsPerCta);
    if (int64_t(blockIdx.x) >= shares) return;
    int64_t u = total * blockIdx.x / shares;
    const int64_t u_end = total * (blockIdx.x + 1) / shares;
    if (u >= before && u < before + mine) {
        int64_t at = before;
        int i = i0;
        for (; i < i1; ++i) {
            const int64_t n = H * share_of(a, i, nullptr).steps;
            if (u < at + n) break;
            at += n;
        }
        s_entry = i;
        s_off = u - at;
    }

    const uint32_t bar = smem_u32(bars);
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sm = smem_u32(smem);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar + 8 * (K_FULL + s), 4);   // the converting warps
            mbar_init(bar + 8 * (V_FULL + s), 4);
            mbar_init(bar + 8 * (K_EMPTY + s), 1);  // products done
            mbar_init(bar + 8 * (V_EMPTY + s), 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(bar + 8 * (S_FULL + g), 2);   // product done, and the issuing thread (which has seen the
                                                    // step's places: K_FULL's release reaches the softmax by it)
            mbar_init(bar + 8 * (P_FULL + g), 4);   // the tile's softmax warps
            mbar_init(bar + 8 * (PV_DONE + g), 1);
        }
        fence_mbar_init();
        s_gone = 0;
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem;  // columns: S0 0, S1 128, O0 256, O1 384
    volatile int *gone = &s_gone;

    int entry = s_entry;
    int64_t off = s_off;
    Share sh = share_of(a, entry, nullptr);
    const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
    const int64_t plane = int64_t(a.layer) * 2 * N, v_plane_bytes = N * B * H * d;
    uint32_t it = 0;        // steps done by this CTA (phases of the K and V barriers)
    uint32_t it_g[2] = {0, 0};  // steps of each tile (phases of its barriers)

    while (u < u_end) {
        while (off >= H * sh.steps) {
            off -= H * sh.steps;
            sh = share_of(a, ++entry, nullptr);
        }
        // the job: KV head h, row tile `tile`, steps [sa, sb)
        const int h = int(off / sh.steps);
        int64_t rest = off - h * sh.steps;
        int tile = 0;
        Tile t = tile_of(a, sh.e, 0);
        while (rest >= t.steps) {
            rest -= t.steps;
            t = tile_of(a, sh.e, ++tile);
        }
        const int sa = int(rest), sb = int(min(int64_t(t.steps), rest + (u_end - u))), n = sb - sa;
        const int64_t job_u0 = u - sa;
        const bool two = t.rows > kTileRows;
        const int pos0 = sh.e.len - sh.e.fresh;
        const int64_t row_base = int64_t(tile) * kJobRows;

        // ---- Q: each row scaled by a power of two into the range of a half (undone in s_cq)
        if (tid == 0) s_nan = 0;
        {
            constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a warp's vector
            const int at = (lane % kLanes) * 8;
#pragma unroll 4
            for (int r = warp * kPer + lane / kLanes; r < kJobRows; r += kThreads / 32 * kPer) {
                float v[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = 0.f;
                if (r < t.rows && at < d) {
                    const int64_t row = row_base + r;
                    load8<TYPE>(static_cast<const uint8_t *>(a.attn.q.data) + (sh.e.row0 + row / G) * a.attn.q.row_stride +
                                    (h * G + row % G) * a.attn.q.head_stride + 2 * at, v);
                }
                float amax = 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x) amax = fmaxf(amax, fabsf(v[x]));
#pragma unroll
                for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const uint32_t ex = (__float_as_uint(amax) >> 23) & 0xffu;
                const bool plain = ex < 2 || ex > 252;
                const float up = plain ? 1.f : __uint_as_float((254u - ex) << 23);
                const float down = plain ? 1.f : __uint_as_float(ex << 23);
                uint4 w;
                w.x = pack2<KVL_TYPE_HALF>(v[0] * up, v[1] * up);
                w.y = pack2<KVL_TYPE_HALF>(v[2] * up, v[3] * up);
                w.z = pack2<KVL_TYPE_HALF>(v[4] * up, v[5] * up);
                w.w = pack2<KVL_TYPE_HALF>(v[6] * up, v[7] * up);
                const int rt = r & (kTileRows - 1), unit = at / 8;
                *reinterpret_cast<uint4 *>(smem + C::kQ + (r / kTileRows) * C::kTileBytes + (unit >> 3) * (kTileRows * 128) +
                                           rt * 128 + (((unit & 7) ^ (rt & 7)) << 4)) = w;
                if (lane % kLanes == 0) s_cq[r] = a.attn.sm_scale * kLog2e * down;
            }
        }
        fence_proxy_async_smem();
        __syncthreads();

        float row_m = -INFINITY, row_l = 0.f;  // of this softmax thread's row
        if (warp >= 8 && warp < 12) {
            // ---- convert K and V
            const int cw = warp - 8;
            constexpr int kLanes = D / 16, kPer = 32 / kLanes, kVecs = 32 / kPer;  // 32 slots a warp
            const int ch = lane % kLanes, rw = lane / kLanes;
            // Lane l looks after group l % 2 of the warp's two in step l / 2 of a batch of 16 steps: its
            // page, place and scales.  The next batch's are fetched while this one is worked on, so
            // no step waits for a table entry or a scale.
            auto place = [&](int s, int &t0, int &nv) -> int32_t {
                t0 = 0;
                nv = 0;
                const int g = t.g0 + (sa + s) * kGroups + cw * 2 + (lane & 1);
                if (g >= t.g1 || s >= n) return -1;
                const int blk = g / per_block, slot = (g - blk * per_block) * kGroup;
                t0 = blk * B + slot;
                nv = min(min(kGroup, B - slot), sh.e.len - t0);
                if (nv <= 0) return -1;
                const int32_t page = sh.e.table[blk];
                if (page < 0 || page >= N) {
                    report(a.report, KVL_ERANGE, entry);
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
            scales(page, ks, vs);
            uint4 kreg[kVecs], vreg[kVecs];
            auto fetch = [&](uint4 (&reg)[kVecs], int s, int base, bool v) {  // step s's codes, of this batch or the next
                const bool ahead = s - base >= 16;
                const uint8_t *half[2];
                int valid[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int from = ((s & 15) << 1) | y;
                    const int32_t pg = __shfl_sync(0xffffffffu, ahead ? page_n : page, from);
                    const int tt = __shfl_sync(0xffffffffu, ahead ? t0n : t0, from);
                    valid[y] = __shfl_sync(0xffffffffu, ahead ? nvn : nv, from);
                    if (ch * 16 >= d) valid[y] = 0;
                    half[y] = codes + (v ? v_plane_bytes : 0) + (((plane + max(pg, 0)) * B + tt % B) * H + h) * d + ch * 16;
                }
#pragma unroll
                for (int x = 0; x < kVecs; ++x) {
                    const int r = (x % (kVecs / 2)) * kPer + rw, y = x / (kVecs / 2);  // slot r of the warp's group y
                    reg[x] = make_uint4(0, 0, 0, 0);
                    if (r < valid[y]) reg[x] = __ldg(reinterpret_cast<const uint4 *>(half[y] + int64_t(r) * H * d));
                }
            };
            auto convert = [&](const uint4 (&reg)[kVecs], uint8_t *dst) {
#pragma unroll
                for (int x = 0; x < kVecs; ++x) {
                    const int r = cw * 32 + x * kPer + rw;
                    const uint32_t w[4] = {reg[x].x, reg[x].y, reg[x].z, reg[x].w};
                    uint4 lo, hi;
                    lo.x = codes_lo<CODE>(w[0]); lo.y = codes_hi<CODE>(w[0]); lo.z = codes_lo<CODE>(w[1]); lo.w = codes_hi<CODE>(w[1]);
                    hi.x = codes_lo<CODE>(w[2]); hi.y = codes_hi<CODE>(w[2]); hi.z = codes_lo<CODE>(w[3]); hi.w = codes_hi<CODE>(w[3]);
                    uint8_t *p = dst + (ch >> 2) * (kTileRows * 128) + r * 128;
                    const int un = (ch & 3) * 2;
                    *reinterpret_cast<uint4 *>(p + ((un ^ (r & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4 *>(p + (((un + 1) ^ (r & 7)) << 4)) = hi;
                }
            };
            fetch(kreg, 0, 0, false);
            fetch(vreg, 0, 0, true);
            int base = 0;
            for (int s = 0; s < n; ++s) {
                if (s - base == 16) {
                    base += 16;
                    page = page_n; t0 = t0n; nv = nvn; ks = ksn; vs = vsn;
                    page_n = place(base + 16 + (lane >> 1), t0n, nvn);
                }
                if (s - base == 4) scales(page_n, ksn, vsn);
                const uint32_t k = it + s, st = k % kStages, ph = (k / kStages) & 1;
                const int two_lanes = (s & 15) << 1;
                const bool here = (lane & ~1) == two_lanes;
                const bool partial = __any_sync(0xffffffffu, here && !(nv == kGroup && t0 >= t.all_lo && t0 + kGroup <= t.all_hi));
                if (!wait_bar(bar + 8 * (K_EMPTY + st), ph ^ 1, gone)) break;
                Places &pl = places[k % kPlaces];
                if (here) {
                    const int g = cw * 2 + (lane & 1);
                    pl.ks[g] = ks;
                    pl.lvs[g] = __log2f(vs);
                    pl.ivs[g] = __fdividef(1.f, vs);
                    pl.t0[g] = t0;
                    pl.nv[g] = nv;
                    pl.partial[cw] = partial;
                }
                convert(kreg, smem + C::kK + st * C::kTileBytes);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (K_FULL + st));
                if (s + 1 < n) fetch(kreg, s + 1, base, false);
                if (CODE == KVL_CODE_FLOAT && partial) {
                    // NaN codes of a step that some rows see in part would reach the others as 0 * NaN:
                    // they leave the products here and come back where the rows are written
                    uint32_t any = 0;
#pragma unroll
                    for (int x = 0; x < kVecs; ++x) {
                        uint32_t w[4] = {vreg[x].x, vreg[x].y, vreg[x].z, vreg[x].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const uint32_t bad = __vcmpeq4(w[y] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            any |= bad;
                            w[y] &= ~bad;
                        }
                        vreg[x] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (any) s_nan = 1;
                }
                if (!wait_bar(bar + 8 * (V_EMPTY + st), ph ^ 1, gone)) break;
                convert(vreg, smem + C::kV + st * C::kTileBytes);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (V_FULL + st));
                if (s + 1 < n) fetch(vreg, s + 1, base, true);
            }
        } else if (warp == 12) {
            // ---- issue the products
            if (lane == 0) {
                constexpr uint32_t kS = instr_desc(kSlots, false), kO = instr_desc(D, true);
                const int tiles = two ? 2 : 1;
                auto scores = [&](int g, uint32_t st) {
                    const uint32_t q = sm + C::kQ + g * C::kTileBytes, k = sm + C::kK + st * C::kTileBytes;
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t o = (x >> 2) * (kTileRows * 128) + (x & 3) * 32;
                        mma_smem(tmem + g * 128, matrix_desc(q + o, 16, 1024), matrix_desc(k + o, 16, 1024), kS, x > 0);
                    }
                    mma_commit(bar + 8 * (S_FULL + g));
                    mbar_arrive(bar + 8 * (S_FULL + g));
                };
                auto values = [&](int g, uint32_t st, bool add) {
                    const uint32_t v = sm + C::kV + st * C::kTileBytes;
#pragma unroll
                    for (int x = 0; x < kSlots / 16; ++x)
                        mma_tmem(tmem + 256 + g * 128, tmem + g * 128 + x * 8,
                                 matrix_desc(v + x * 2048, kTileRows * 128, 1024), kO, add || x > 0);
                    mma_commit(bar + 8 * (PV_DONE + g));
                };
                bool ok = true;
                for (int s = 0; s <= n && ok; ++s) {
                    const uint32_t k = it + s, st = k % kStages;
                    const uint32_t kp = k - 1, sp = kp % kStages;
                    for (int g = 0; g < tiles && ok; ++g) {
                        if (s > 0) {
                            ok = wait_bar(bar + 8 * (P_FULL + g), (it_g[g] + s - 1) & 1, gone) &&
                                 (g > 0 || wait_bar(bar + 8 * (V_FULL + sp), (kp / kStages) & 1, gone));
                            if (!ok) break;
                            tmem_fence_after();
                            values(g, sp, s > 1);
                            if (g == tiles - 1) mma_commit(bar + 8 * (V_EMPTY + sp));
                        }
                        if (s < n) {
                            if (g == 0 && !(ok = wait_bar(bar + 8 * (K_FULL + st), (k / kStages) & 1, gone))) break;
                            tmem_fence_after();
                            scores(g, st);
                            if (g == tiles - 1) mma_commit(bar + 8 * (K_EMPTY + st));
                        }
                    }
                }
            }
            __syncwarp();
        } else if (warp < 8 && (warp < 4 || two)) {
            // ---- softmax: row r of the job, TMEM lane r % 128
            const int g = warp >> 2, r = tid & 255;
            const uint32_t lanes = uint32_t(warp & 3) << 21;  // lane 32 (warp % 4), in bits 16 and up
            const uint32_t ts = tmem + lanes + g * 128, to = tmem + lanes + 256 + g * 128;
            const int pos = pos0 + int((row_base + r) / G);
            int hi = a.attn.causal ? min(sh.e.len, pos + 1) : sh.e.len;
            int lo = a.attn.window > 0 ? max(0, pos - a.attn.window + 1) : 0;
            if (r >= t.rows) { lo = t.all_lo; hi = t.all_hi; }
            const float cq = s_cq[r];
            constexpr uint32_t kHidden = 0xff800000u;  // -infinity
            bool ok = true;
            for (int s = 0; s < n; ++s) {
                const uint32_t ph = (it_g[g] + s) & 1;
                ok = __all_sync(0xffffffffu, wait_bar(bar + 8 * (S_FULL + g), ph, gone));
                if (!ok) break;
                tmem_fence_after();
                const Places &pl = places[(it + s) % kPlaces];
                auto hide = [&](uint32_t (&x)[32], int gi) {  // scores of groups gi, gi + 1 that the row does not see
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int first = max(lo - pl.t0[gi + y], 0), past = min(hi - pl.t0[gi + y], pl.nv[gi + y]);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e < first || e >= past) x[16 * y + e] = kHidden;
                    }
                };
                const bool whole = !(pl.partial[0] | pl.partial[1] | pl.partial[2] | pl.partial[3]);
                // the step's largest x: scales are not negative, so a group's largest comes from its
                // largest score
                float big = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld32(ts + 32 * c, x);
                    tmem_wait_ld();
                    if (!whole) hide(x, 2 * c);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = __uint_as_float(x[16 * y]);
#pragma unroll
                        for (int e = 1; e < 16; ++e) top = fmaxf(top, __uint_as_float(x[16 * y + e]));
                        const float z = fmaf(top, pl.ks[2 * c + y] * cq, pl.lvs[2 * c + y]);
                        if (top != -INFINITY) big = fmaxf(big, z);
                    }
                }
                const bool grow = big > row_m + kSlack || (row_m == -INFINITY && big > -INFINITY);
                if (__any_sync(0xffffffffu, grow)) {
                    const float m = grow ? big : row_m;
                    const float f = grow ? exp2_of(row_m - m) : 1.f;  // 0 from a first maximum
                    row_l *= f;
                    row_m = m;
                    if (s > 0) {
                        ok = __all_sync(0xffffffffu, wait_bar(bar + 8 * (PV_DONE + g), ph ^ 1, gone));
                        if (!ok) break;
                        tmem_fence_after();
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t x[32];
                            tmem_ld32(to + 32 * c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                            tmem_st32(to + 32 * c, x);
                        }
                    }
                }
                const float ref = row_m == -INFINITY ? 0.f : row_m;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32], p[16];
                    tmem_ld32(ts + 32 * c, x);
                    tmem_wait_ld();
                    if (!whole) hide(x, 2 * c);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float f = pl.ks[2 * c + y] * cq, b = pl.lvs[2 * c + y] - ref;
                        float sum = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            // a hidden score is -infinity: its weight has to be 0 whatever f and b are
                            float w0 = exp2_of(fmaf(__uint_as_float(x[16 * y + e]), f, b));
                            float w1 = exp2_of(fmaf(__uint_as_float(x[16 * y + e + 1]), f, b));
                            if (!whole) {
                                if (x[16 * y + e] == kHidden) w0 = 0.f;
                                if (x[16 * y + e + 1] == kHidden) w1 = 0.f;
                            }
                            sum += w0 + w1;
                            p[8 * y + e / 2] = pack2<KVL_TYPE_HALF>(w0, w1);
                        }
                        if (sum != 0.f) row_l = fmaf(sum, pl.ivs[2 * c + y], row_l);
                    }
                    tmem_st16(ts + 16 * c, p);
                }
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (P_FULL + g));
            }
            if (ok) {
                ok = __all_sync(0xffffffffu, wait_bar(bar + 8 * (PV_DONE + g), (it_g[g] + n - 1) & 1, gone));
                tmem_fence_after();
            }
            // ---- the row's result, or its part
            const bool complete = sa == 0 && sb == t.steps;
            uint32_t nan_at[D / 32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) nan_at[c] = 0;
            if (ok && CODE == KVL_CODE_FLOAT && *const_cast<volatile int *>(&s_nan) && r < t.rows) {
                // elements that a NaN code of a seen token reaches, from the steps that were cleared
                for (int gi = t.g0 + sa * kGroups; gi < min(t.g1, t.g0 + sb * kGroups); ++gi) {
                    const int blk = gi / per_block, slot = (gi - blk * per_block) * kGroup, t0 = blk * B + slot;
                    const int nv = min(min(kGroup, B - slot), sh.e.len - t0);
                    const int32_t page = sh.e.table[blk];
                    if (page < 0 || page >= N) continue;
                    for (int e = 0; e < nv; ++e) {
                        if (t0 + e < lo || t0 + e >= hi) continue;
                        const uint8_t *p = codes + v_plane_bytes + (((plane + page) * B + slot + e) * H + h) * d;
                        for (int x = 0; x < d; ++x)
                            if ((p[x] & 0x7f) == 0x7f) {
#pragma unroll
                                for (int c = 0; c < D / 32; ++c)
                                    if (c == x / 32) nan_at[c] |= 1u << (x & 31);
                            }
                    }
                }
            }
            const int64_t row = row_base + r;
            const float inv = row_l == 0.f ? 0.f : 1.f / row_l;
            float *part = a.parts + (int64_t(blockIdx.x) * 2 + (sa == 0 ? 1 : 0)) * C::kPartFloats;
            uint8_t *dst = static_cast<uint8_t *>(a.attn.out.data) + (sh.e.row0 + row / G) * a.attn.out.row_stride +
                           (h * G + row % G) * a.attn.out.head_stride;
            if (ok) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
                    tmem_ld32(to + 32 * c, x);
                    tmem_wait_ld();
                    if (nan_at[c]) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (nan_at[c] >> e & 1u) x[e] = 0x7fffffffu;
                    }
                    if (r < t.rows) {
                        if (complete) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float v[8];
#pragma unroll
                                for (int y = 0; y < 8; ++y) v[y] = __uint_as_float(x[8 * e + y]) * inv;
                                if (32 * c + 8 * e < d) store8<TYPE>(dst + 2 * (32 * c + 8 * e), v);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4 *>(part + 2 * kJobRows + (int64_t(8 * c + e) * kJobRows + r) * 4) =
                                    make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                        }
                    }
                }
                if (r < t.rows) {
                    if (!complete) {
                        part[r] = row_m;
                        part[kJobRows + r] = row_l;
                    } else if (a.attn.lse) {
                        a.attn.lse[(sh.e.row0 + row / G) * a.attn.n_heads + h * G + row % G] =
                            row_l == 0.f ? -INFINITY : (row_m + __log2f(row_l)) * (1.f / kLog2e);
                    }
                }
            }
            tmem_fence_before();
        }
        it += n;
        it_g[0] += n;
        if (two) it_g[1] += n;
        if (!(sa == 0 && sb == t.steps)) {
            // parts of this job: shares first .. last; the one that arrives last joins them
            const int first = int(((job_u0 + 1) * shares - 1) / total);
            const int last = int(((job_u0 + t.steps) * shares - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = !*gone && atomicAdd(&a.counters[first], 1u) == uint32_t(last - first);
            __syncthreads();
            if (s_last) {
                __threadfence();
                if (tid == 0) a.counters[first] = 0;
                const int r = tid & (kJobRows - 1);
                if (r < t.rows) {
                    auto part_of = [&](int b) { return a.parts + (int64_t(b) * 2 + (b == first)) * C::kPartFloats; };
                    float big = -INFINITY, sum = 0.f;
                    for (int b = first; b <= last; ++b) big = fmaxf(big, __ldcg(part_of(b) + r));
                    for (int b = first; b <= last; ++b) {
                        const float mb = __ldcg(part_of(b) + r);
                        sum += __ldcg(part_of(b) + kJobRows + r) * (mb == -INFINITY ? 0.f : exp2_of(mb - big));
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const int64_t row = row_base + r;
                    const int head = int(h * G + row % G);
                    uint8_t *dst = static_cast<uint8_t *>(a.attn.out.data) + (sh.e.row0 + row / G) * a.attn.out.row_stride +
                                   head * a.attn.out.head_stride;
#pragma unroll 4
                    for (int e = (tid / kJobRows) * 2; e < D / 4; e += 4) {  // 8 elements: two vectors of 4
                        float v[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x) v[x] = 0.f;
                        for (int b = first; b <= last; ++b) {
                            const float *p = part_of(b);
                            const float mb = __ldcg(p + r);
                            const float f = mb == -INFINITY ? 0.f : exp2_of(mb - big);
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float4 y = __ldcg(reinterpret_cast<const float4 *>(p + 2 * kJobRows) + int64_t(e + x) * kJobRows + r);
                                v[4 * x] += y.x * f; v[4 * x + 1] += y.y * f; v[4 * x + 2] += y.z * f; v[4 * x + 3] += y.w * f;
                            }
                        }
#pragma unroll
                        for (int x = 0; x < 8; ++x) v[x] *= inv;
                        if (4 * e < d) store8<TYPE>(dst + 8 * e, v);
                    }
                    if (a.attn.lse && tid < kJobRows)
                        a.attn.lse[(sh.e.row0 + row / G) * a.attn.n_heads + head] =
                            sum == 0.f ? -INFINITY : (big + __log2f(sum)) * (1.f / kLog2e);
                }
            }
        }
        __syncthreads();  // Q and tensor memory are free again
        tmem_fence_after();
        if (*gone) break;
        off += n;
        u += n;
    }
    if (*gone) {
        if (tid == 0) report(a.report, KVL_ETIMEOUT, blockIdx.x);
        if (warp == 12 && lane == 0) {  // let the products in flight end (bounded) before their memory goes
            mbar_inval(bar + 8 * P_FULL);
            mbar_init(bar + 8 * P_FULL, 1);
            fence_mbar_init();
            mma_commit(bar + 8 * P_FULL);
            mbar_wait_bounded(bar + 8 * P_FULL, 0);
        }
    }
    __syncthreads();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int CODE, int TYPE, int D>
kvl_status launch_chunk(const AttendArgs &a, int sms, void *stream)
{
    static std::atomic<unsigned long long> ready[kMaxDevices];
    if (!allow_smem(attend_chunk_kernel<CODE, TYPE, D>, ready, Chunk<D>::kSmem)) return KVL_ECUDA;
    attend_chunk_kernel<CODE, TYPE, D><<<sms, kThreads, Chunk<D>::kSmem, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}

template <int CODE, int TYPE>
kvl_status launch_chunk_dim(const AttendArgs &a, int sms, void *stream)
{
    return a.cache.head_dim <= 64 ? launch_chunk<CODE, TYPE, 64>(a, sms, stream) : launch_chunk<CODE, TYPE, 128>(a, sms, stream);
}

}  // namespace

size_t attend_chunk_part_bytes(int head_dim)
{
    return head_dim > 128 ? 0 : size_t(2) * kJobRows * ((head_dim <= 64 ? 64 : 128) + 2) * sizeof(float);
}

kvl_status launch_attend_chunk(const AttendArgs &a, int sms, void *stream)
{
    const bool bf = a.attn.type == KVL_TYPE_BFLOAT;
    if (a.cache.code_type == KVL_CODE_FLOAT)
        return bf ? launch_chunk_dim<KVL_CODE_FLOAT, KVL_TYPE_BFLOAT>(a, sms, stream)
                  : launch_chunk_dim<KVL_CODE_FLOAT, KVL_TYPE_HALF>(a, sms, stream);
    return bf ? launch_chunk_dim<KVL_CODE_INT, KVL_TYPE_BFLOAT>(a, sms, stream)
              : launch_chunk_dim<KVL_CODE_INT, KVL_TYPE_HALF>(a, sms, stream);
}

}  // namespace kvl

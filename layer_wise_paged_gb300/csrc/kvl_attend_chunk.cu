// kvl_attend_chunk.cu -- attention of many rows a sequence: prompts and their chunks.
//
// 4 d operations for each (row, visible token), which is above the tensor cores' floor for prompts; bound
// by the chain product, softmax, product of a tile (512 tokens of 32 heads on 31,232: 223 us where the
// products alone take 135; a tile's turn of 3,700 cycles is 1,700 of softmax, 1,230 of products and 800 of
// handing over, and at d = 128 tensor memory has no columns for a second S of 128 slots).  One CTA an SM takes
// 256 rows of one KV head (query heads of the head times tokens), two accumulator tiles of 128,
// and walks the tokens 128 slots (8 groups) at a time:
//   warps 0-3, 4-7   softmax of tile 0, tile 1: a thread a row.  S comes from tensor memory, P goes
//                    back over it as halves, O is rescaled in place when the maximum has outgrown
//                    the reference (kSlack).  The first warp of each issues its tile's products:
//                    O += P V of the step (P in tensor memory, V token-major), then S = Q K^T of
//                    the next (both in shared memory, K-major); the tiles take turns, so one's
//                    softmax runs under the other's products;
//   warps 8-11       read K and V codes from the pages, convert them to halves (exact) and lay
//                    them out in shared memory for the tensor cores (128-byte swizzle), two
//                    stages each, with the groups' scales and places beside them; between jobs
//                    they find the next one and lay out its Q.
// A converted K or V stage serves 256 rows, which is what keeps the conversion (16 bytes in, 32
// out a vector) small beside the products.
//
// Every wait on a memory barrier is bounded, and a warp's lanes go on or give up together: past the limit a
// flag is raised, the report says KVL_ETIMEOUT, every role leaves in an order that leaves no warp waiting at a
// named barrier (kvl_attend_meet.cuh), and the tensor memory is given back.
#include <type_traits>

#include "kvl_attend.cuh"
#include "kvl_attend_meet.cuh"

namespace kvl {
namespace {

constexpr int kThreads = 384;  // 8 softmax warps, 4 converting: 168 registers a thread
constexpr int kTileRows = 128;
constexpr int kJobRows = 2 * kTileRows;
constexpr int kSlots = 128;                 // slots of a step
constexpr int kGroups = kSlots / kGroup;    // 8
constexpr int kStages = 2;
constexpr int kPlaces = 4;                  // steps whose scales are kept (see place_full)
constexpr int kBatch = 512;                 // entries whose steps are held at a time
// Units of a share: a job's steps, and kJobCost before them for starting it (finding it, loading Q,
// filling the pipeline; prompts of a few jobs a CTA: 355 us, with 4 374, with 8 366, with none 520).
constexpr int kJobCost = 6;
constexpr int kStepsPerCta = kJobCost + 2;  // a share is at least this many units

// Scales and places of a step's groups; partial[w]: some row sees only a part of the two groups that
// converting warp w filled.
struct alignas(16) Places {
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
enum Bar { K_FULL = 0, K_EMPTY = 2, V_FULL = 4, V_EMPTY = 6, S_FULL = 8, PV_DONE = 10, LEAVE = 12, BARS = 13 };

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

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// Products, issued by the elected lane of a converged warp.
__device__ __forceinline__ void mma_smem(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(uint32_t(add)), "r"(one)
        : "memory");
}

__device__ __forceinline__ void mma_tmem(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(uint32_t(add)), "r"(one)
        : "memory");
}

// Arrives on the barrier when the products that the elected lane has issued so far have ended.
__device__ __forceinline__ void mma_commit(uint32_t one, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
        : "memory");
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

__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
}

__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
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

// Named barriers (kvl_attend_meet.cuh).  They are not in shared memory, where an access takes 200 cycles
// while products stream their operands.
struct Meet {
    template <int N>
    __device__ __forceinline__ void wait(int id) const { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory"); }
    template <int N>
    __device__ __forceinline__ void arrive(int id) const { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(N) : "memory"); }
};

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two floats in one register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair_of(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 split_pair(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Bounded wait that also leaves when another role has given up.  The limit (kWaitLimitNs at the
// highest clock) is looked at every 256 tries: reading the global timer on the way in cost up to a
// thousand cycles after the barrier had completed.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *gone)
{
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t tries = 1; !mbar_try_wait(bar, parity); ++tries) {
        if (tries & 255) continue;
        if (*gone) return false;
        if (clock64() - t0 > 2 * static_cast<long long>(kWaitLimitNs)) {
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

__device__ __forceinline__ Tile tile_of(const AttendArgs &a, int32_t len, int32_t fresh, int tile)
{
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup, G = a.attn.n_heads / a.cache.n_kv_heads;
    Tile t;
    const uint32_t row0 = uint32_t(tile) * kJobRows;
    t.rows = min(kJobRows, int32_t(uint32_t(fresh) * G - row0));
    const int pos0 = len - fresh;
    const int first = pos0 + int(row0 / uint32_t(G)), last = pos0 + int((row0 + t.rows - 1) / uint32_t(G));
    const int hi = a.attn.causal ? min(len, last + 1) : len;
    const int lo = first_seen(a, first);
    t.all_hi = a.attn.causal ? min(len, first + 1) : len;
    t.all_lo = first_seen(a, last);
    t.g0 = t.g1 = 0;
    if (hi > lo) {
        t.g0 = group_of(lo, B, per_block);
        t.g1 = group_of(hi - 1, B, per_block) + 1;
    }
    t.steps = max(1, (t.g1 - t.g0 + kGroups - 1) / kGroups);
    return t;
}

__device__ __forceinline__ int32_t tiles_of(const AttendArgs &a, const Entry &e)
{
    const int32_t rows = e.fresh * (a.attn.n_heads / a.cache.n_kv_heads);  // the host has bounded n_rows
    return rows > a.max_rows ? (rows + kJobRows - 1) / kJobRows : 0;
}

// Units of one KV head of an entry, all tiles: a warp's lanes take a tile each.
__device__ __forceinline__ uint32_t warp_units(const AttendArgs &a, int32_t len, int32_t fresh, int32_t tiles, int lane)
{
    uint64_t n = 0;
    for (int t = lane; t < tiles; t += 32) n += tile_of(a, len, fresh, t).steps + kJobCost;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return uint32_t(min(n, kMostUnits));
}

// Where a CTA stands in its share, and the job it works on: in shared memory, so that the roles' loops
// hold only what they use in registers.
struct Job {
    Cut cut;
    uint32_t u, u_end, off;   // next unit, the share's end, units of the entry before u
    uint32_t u0;              // the unit of the job's first step
    int32_t taken;            // units of the job in this share
    int32_t row_base;         // the tile's first row
    Entry e;
    Tile t;
    int32_t entry, h, sa, n;  // KV head; steps [sa, sa + n) of the tile
    int32_t pos0;             // position of the entry's first fresh row
    int32_t two;              // the second half tile has rows
    int32_t half;             // of s_cq
    uint32_t it, it_g[2];     // steps done by this CTA, and of each half tile: the barriers' phases
    bool complete;            // the share holds the whole job
};

// The job that holds unit job.u, of which this share has the units from there on; n = 0 where they are
// only units before its steps.  Called by one whole warp.
__device__ __forceinline__ void next_job(const AttendArgs &a, Job &job, int lane)
{
    const int H = a.cache.n_kv_heads, B = a.cache.block_tokens;
    uint32_t off = job.off;
    int entry = job.entry;
    Entry e = load_entry(a.seqs, B, entry, nullptr);
    int32_t tiles = tiles_of(a, e);
    uint32_t units = warp_units(a, e.len, e.fresh, tiles, lane);
    while (off >= H * units) {
        off -= H * units;
        e = load_entry(a.seqs, B, ++entry, nullptr);
        tiles = tiles_of(a, e);
        units = warp_units(a, e.len, e.fresh, tiles, lane);
    }
    const int h = int(off / units);
    uint32_t rest = off - h * units;
    // the tile whose units hold `rest`: 32 tiles at a time
    int tile = 0;
    for (int base = 0; base < tiles; base += 32) {
        const int n = base + lane < tiles ? tile_of(a, e.len, e.fresh, base + lane).steps + kJobCost : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, rest < uint32_t(sum));
        if (past) {
            const int l = __ffs(past) - 1;
            tile = base + l;
            rest -= __shfl_sync(0xffffffffu, sum - n, l);
            break;
        }
        rest -= __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
        const Tile t = tile_of(a, e.len, e.fresh, tile);
        const uint32_t taken = min(t.steps + kJobCost - rest, job.u_end - job.u);
        job.off = off;
        job.entry = entry;
        job.e = e;
        job.t = t;
        job.h = h;
        job.sa = max(0, int(rest) - kJobCost);
        job.n = max(0, int(rest + taken) - kJobCost) - job.sa;
        job.taken = int(taken);
        job.u0 = job.u - rest + kJobCost;
        job.row_base = tile * kJobRows;
        job.pos0 = e.len - e.fresh;
        job.two = t.rows > kTileRows;
        job.complete = job.n == t.steps;
    }
}

// A part of `job` has come, or will not come; by one thread.  Whether it is to join the parts.
__device__ __forceinline__ bool arrive_part(const AttendArgs &a, const Job &job, bool no_result)
{
    const uint32_t first = job.cut.share_of(job.u0), last = job.cut.share_of(job.u0 + job.t.steps - 1);
    const Arrival x = arrival(atomicAdd(&a.counters[first], no_result ? 1 + kNoResult : 1), last - first + 1, no_result);
    if (x.last) a.counters[first] = 0;
    return x.join;
}

// The jobs of the share that have not been begun will not come: `job` (if n > 0) and those after it.  By one
// whole warp of a CTA that gives up.  (Not inlined: its code in the roles' would cost 3 us of 350.)
__device__ __noinline__ void arrive_without_result(const AttendArgs &a, Job &job, int lane)
{
    while (true) {
        if (lane == 0 && job.n > 0 && !job.complete) arrive_part(a, job, true);
        const uint32_t u = job.u + job.taken, off = job.off + job.taken;
        __syncwarp();
        if (u >= job.u_end) break;
        if (lane == 0) {
            job.u = u;
            job.off = off;
        }
        __syncwarp();
        next_job(a, job, lane);
        __syncwarp();
    }
}

// The products of tile g from K or V stage st, issued by a whole warp of which lane `one` is elected.
// Kept short: the roles' loops together just fit the instruction cache, and with four copies of
// these (a tile and stage each) the 512 rows on 31,232 took 295 us instead of 270.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t one, uint32_t sm, int g, uint32_t st)
{
    using C = Chunk<D>;
    uint64_t q = matrix_desc(sm + C::kQ + g * C::kTileBytes, 16, 1024), k = matrix_desc(sm + C::kK + st * C::kTileBytes, 16, 1024);
#pragma unroll 1
    for (int x = 0; x < D / 64; ++x) {
#pragma unroll
        for (int y = 0; y < 4; ++y) mma_smem(one, g * 128, q + 2 * y, k + 2 * y, instr_desc(kSlots, false), x + y > 0);
        q += kTileRows * 128 >> 4;
        k += kTileRows * 128 >> 4;
    }
}

template <int D>
__device__ __forceinline__ void issue_values(uint32_t one, uint32_t sm, int g, uint32_t st, bool add)
{
    using C = Chunk<D>;
    uint64_t v = matrix_desc(sm + C::kV + st * C::kTileBytes, kTileRows * 128, 1024);
    uint32_t p = g * 128;
#pragma unroll 1
    for (int x = 0; x < kSlots / 64; ++x) {
#pragma unroll
        for (int y = 0; y < 4; ++y) mma_tmem(one, 256 + g * 128, p + y * 8, v + y * (2048 >> 4), instr_desc(D, true), add || x + y > 0);
        p += 32;
        v += 4 * 2048 >> 4;
    }
}

template <int CODE, int TYPE, int D>
__global__ void __launch_bounds__(kThreads, 1) attend_chunk_kernel(const __grid_constant__ AttendArgs a)
{
    using C = Chunk<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long bars[BARS];
    __shared__ Places places[kPlaces];
    __shared__ float s_cq[2][kJobRows];
    __shared__ uint32_t s_units[kBatch];
    __shared__ Job job, next;
    __shared__ int s_last, s_gone, s_nan;
    __shared__ uint32_t s_tmem;

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int G = a.attn.n_heads / H, per_block = (B + kGroup - 1) / kGroup;
    const int64_t N = a.cache.pool_blocks;

    // ---- this CTA's share of the steps: the entries' steps a batch at a time (entry i of a batch by
    // warp i % 12, its tiles by the lanes), their sum, then the entry that holds the share's first
    uint64_t before = 0;
    uint32_t u = 0;
    Cut cut;
    for (int pass = 0; pass < 2; ++pass) {
        for (int base = 0; base < a.seqs.n_seq; base += kBatch) {
            const int n = min(kBatch, a.seqs.n_seq - base);
            if (pass == 0 || a.seqs.n_seq > kBatch) {
                __syncthreads();
                for (int i = warp; i < n; i += kThreads / 32) {
                    const Entry e = load_entry(a.seqs, B, base + i, pass == 0 && blockIdx.x == 0 && lane == 0 ? a.report : nullptr);
                    const uint32_t units = warp_units(a, e.len, e.fresh, tiles_of(a, e), lane);
                    if (lane == 0) s_units[i] = units;
                }
                __syncthreads();
            }
            // 32 lanes scan the batch; every warp does, and finds the same
            for (int i = 0; i < n; i += 32) {
                uint64_t x = i + lane < n ? uint64_t(s_units[i + lane]) * H : 0, sum = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                if (pass == 1) {
                    const unsigned past = __ballot_sync(0xffffffffu, u < before + sum);
                    if (past) {
                        const int l = __ffs(past) - 1;
                        const uint32_t at = uint32_t(before + __shfl_sync(0xffffffffu, sum - x, l));
                        if (tid == 0) {
                            job.entry = base + i + l;
                            job.off = u - at;
                            job.u = u;
                            job.u_end = cut.start(blockIdx.x + 1);
                            job.cut = cut;
                            job.it = job.it_g[0] = job.it_g[1] = 0;
                            job.n = job.taken = job.two = job.half = 0;
                        }
                        base = a.seqs.n_seq;  // found: leave both loops
                        break;
                    }
                }
                before += __shfl_sync(0xffffffffu, sum, 31);
            }
        }
        if (pass == 0) {
            if (before == 0 || before >= kMostUnits) {
                if (before && blockIdx.x == 0 && tid == 0) report(a.report, KVL_ERANGE, a.seqs.n_seq);
                return;
            }
            cut = Cut(uint32_t(before), min(gridDim.x, (uint32_t(before) + kStepsPerCta - 1) / kStepsPerCta));
            if (blockIdx.x >= cut.shares) return;
            u = cut.start(blockIdx.x);
            before = 0;
        }
    }

    const uint32_t bar = smem_u32(bars);
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sm = smem_u32(smem);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar + 8 * (K_FULL + s), 4);   // the converting warps
            mbar_init(bar + 8 * (V_FULL + s), 4);
            mbar_init(bar + 8 * (K_EMPTY + s), 2);  // both tiles' products done
            mbar_init(bar + 8 * (V_EMPTY + s), 2);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(bar + 8 * (S_FULL + g), 2);   // product done, and the issuing thread (which has seen the
                                                    // step's places: K_FULL's release reaches the softmax by it)
            mbar_init(bar + 8 * (PV_DONE + g), 1);
        }
        mbar_init(bar + 8 * LEAVE, 1);
        fence_mbar_init();
        s_gone = 0;
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    constexpr uint32_t tmem = 0;  // columns: S0 0, S1 128, O0 256, O1 384
    if (s_tmem != 0) {            // all 512 columns were asked for: they begin at 0
        if (tid == 0) report(a.report, KVL_ECUDA, blockIdx.x);
        if (warp == 8) arrive_without_result(a, job, lane);
        if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(s_tmem) : "memory");
        return;
    }
    volatile int *gone = &s_gone;
    const Meet meet;

    const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
    const int64_t plane = int64_t(a.layer) * 2 * N, v_plane_bytes = N * B * H * d;

    // Q of the job in `next` to its place, by the converting warps: each row scaled by a power of two into
    // the range of a half (undone in s_cq), as in attend_rows.  All rows come by asynchronous copies into the (free) K stages,
    // each vector to the thread that takes it on from there.
    auto load_q = [&] {
        const int cw = warp - 8, rows = next.t.rows, h = next.h, row0 = next.e.row0, row_base = next.row_base;
        float *cq = s_cq[next.half];
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a warp's vector
        const int at = (lane % kLanes) * 8;
        const int turns = (next.two ? kJobRows : kTileRows) / (4 * kPer);
        const uint32_t stage = sm + C::kK + (tid & 127) * 16;
#pragma unroll 2
        for (int x = 0; x < turns; ++x) {
            const int r = (cw + x * 4) * kPer + lane / kLanes;
            const bool ok = r < rows && at < d;
            const uint32_t row = ok ? row_base + r : 0, tok = row / uint32_t(G);
            copy_async16(stage + x * 2048,
                         static_cast<const uint8_t *>(a.attn.q.data) + int64_t(row0 + tok) * a.attn.q.row_stride +
                             int64_t(h * G + row - tok * G) * a.attn.q.head_stride + (ok ? 2 * at : 0), ok);
        }
        copy_async_commit();
        copy_async_wait<0>();
#pragma unroll 4
        for (int x = 0; x < turns; ++x) {
            const int r = (cw + x * 4) * kPer + lane / kLanes;
            const uint4 raw = ld_shared_v4(stage + x * 2048);
            float v[8];
            load8<TYPE>(reinterpret_cast<const uint8_t *>(&raw), v);
            float amax = 0.f;
#pragma unroll
            for (int y = 0; y < 8; ++y) amax = fmaxf(amax, fabsf(v[y]));
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
            if (lane % kLanes == 0) cq[r] = a.attn.sm_scale * kLog2e * down;
        }
        fence_proxy_async_smem();
    };

    // Each turn: the job's steps, beside which the converting warps find the next job and load its Q as
    // soon as the last product that reads Q is done, so that only the first job (the first turn has no
    // steps) waits for its Q.
    while (true) {
        if (warp >= 8) {
            // ---- convert K and V
            const int cw = warp - 8, n = job.n, h = job.h, len = job.e.len;
            const uint32_t it = job.it;
            if (n > 0) {
            const int32_t *table = job.e.table;
            const int g0 = job.t.g0 + job.sa * kGroups, g1 = job.t.g1, all_lo = job.t.all_lo, all_hi = job.t.all_hi;
            constexpr int kPer = 512 / D, kVecs = 32 / kPer;  // rows of a warp's vector, vectors of its 32 slots
            // 8 lanes of a shared-memory phase write 4 chunks of an even and of an odd row: with the
            // swizzle, 8 different 16-byte columns
            const int ch = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0), rw = D == 128 ? (lane >> 2) & 3 : lane >> 2;
            // Lane l looks after group l % 2 of the warp's two in step l / 2 of a batch of 16 steps: its
            // page, place and scales.  The next batch's are fetched while this one is worked on, so
            // no step waits for a table entry or a scale.
            auto place = [&](int s, int &t0, int &nv) -> int32_t {
                t0 = 0;
                nv = 0;
                const int g = g0 + s * kGroups + cw * 2 + (lane & 1);
                if (g >= g1 || s >= n) return -1;
                const int blk = g / per_block, slot = (g - blk * per_block) * kGroup;
                t0 = blk * B + slot;
                nv = min(min(kGroup, B - slot), len - t0);
                if (nv <= 0) return -1;
                const int32_t page = table[blk];
                if (page < 0 || page >= N) {
                    report(a.report, KVL_ERANGE, job.entry);
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
            // This lane's place in the warp's two groups of a step (of this batch or the next), and its codes.
            const uint8_t *half[2];
            int valid[2];
            auto look = [&](int s, int base) {
                const bool ahead = s - base >= 16;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int from = ((s & 15) << 1) | y;
                    const int32_t pg = __shfl_sync(0xffffffffu, ahead ? page_n : page, from);
                    const int tt = __shfl_sync(0xffffffffu, ahead ? t0n : t0, from);
                    valid[y] = __shfl_sync(0xffffffffu, ahead ? nvn : nv, from);
                    if (ch * 16 >= d) valid[y] = 0;
                    half[y] = codes + (((plane + max(pg, 0)) * B + tt % B) * H + h) * d + ch * 16;
                }
            };
            auto fetch = [&](uint4 (&reg)[kVecs], int64_t plane_bytes) {
#pragma unroll
                for (int x = 0; x < kVecs; ++x) {
                    const int r = (x % (kVecs / 2)) * kPer + rw, y = x / (kVecs / 2);  // slot r of the warp's group y
                    reg[x] = make_uint4(0, 0, 0, 0);
                    if (r < valid[y]) reg[x] = __ldg(reinterpret_cast<const uint4 *>(half[y] + plane_bytes + int64_t(r) * H * d));
                }
            };
            auto convert = [&](const uint4 (&reg)[kVecs], uint8_t *dst) {
#pragma unroll
                for (int x = 0; x < kVecs; ++x) {
                    const int r = cw * 32 + x * kPer + rw;
                    const uint32_t w[4] = {reg[x].x, reg[x].y, reg[x].z, reg[x].w};
                    uint4 lo, hi;
                    codes_of<CODE>(w[0], lo.x, lo.y);
                    codes_of<CODE>(w[1], lo.z, lo.w);
                    codes_of<CODE>(w[2], hi.x, hi.y);
                    codes_of<CODE>(w[3], hi.z, hi.w);
                    uint8_t *p = dst + (ch >> 2) * (kTileRows * 128) + r * 128;
                    const int un = (ch & 3) * 2;
                    *reinterpret_cast<uint4 *>(p + ((un ^ (r & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4 *>(p + (((un + 1) ^ (r & 7)) << 4)) = hi;
                }
            };
            look(0, 0);
            fetch(kreg, 0);
            fetch(vreg, v_plane_bytes);
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
                const bool partial = __any_sync(0xffffffffu, here && !(nv == kGroup && t0 >= all_lo && t0 + kGroup <= all_hi));
                if (!__all_sync(0xffffffffu, wait_bar(bar + 8 * (K_EMPTY + st), ph ^ 1, gone))) break;  // (the lanes go or stay together)
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
                if (s + 1 < n) {
                    look(s + 1, base);
                    fetch(kreg, 0);
                }
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
                if (!__all_sync(0xffffffffu, wait_bar(bar + 8 * (V_EMPTY + st), ph ^ 1, gone))) break;
                convert(vreg, smem + C::kV + st * C::kTileBytes);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (V_FULL + st));
                if (s + 1 < n) fetch(vreg, v_plane_bytes);
            }
            }
            // the stages of the two steps that would come next are free, so all of K's readers are done
            const uint32_t k0 = it + n, k1 = k0 + 1;
            const bool free = __all_sync(0xffffffffu, wait_bar(bar + 8 * (K_EMPTY + k0 % kStages), ((k0 / kStages) & 1) ^ 1, gone) &&
                                                          wait_bar(bar + 8 * (K_EMPTY + k1 % kStages), ((k1 / kStages) & 1) ^ 1, gone));
            if (warp == 8) {
                if (lane == 0) {
                    next = job;
                    next.it += n;
                    next.it_g[0] += n;
                    if (job.two) next.it_g[1] += n;
                    next.half ^= 1;
                    next.n = 0;
                }
                __syncwarp();
                while (free) {
                    const uint32_t u0 = next.u + next.taken, off = next.off + next.taken;
                    __syncwarp();
                    if (u0 >= next.u_end) break;
                    if (lane == 0) {
                        next.u = u0;
                        next.off = off;
                    }
                    __syncwarp();
                    next_job(a, next, lane);
                    __syncwarp();
                    if (next.n > 0) break;  // (its steps may be the next share's)
                }
            }
            meet.wait<128>(kQBar);
            if (free && next.n > 0) load_q();
        } else if (job.n > 0 && (warp < 4 || job.two)) {
            // ---- softmax: row r of the job, TMEM lane r % 128
            const int g = warp >> 2, r = tid & 255;  // (uniform: warp is)
            const uint32_t lanes = uint32_t(warp & 3) << 21;  // lane 32 (warp % 4), in bits 16 and up
            const uint32_t ts = tmem + lanes + g * 128, to = tmem + lanes + 256 + g * 128;
            const uint32_t it = job.it, it_g = g ? job.it_g[1] : job.it_g[0];
            const int n = job.n;
            int lo, hi;
            {
                const int pos = job.pos0 + int(uint32_t(job.row_base + r) / uint32_t(G)), len = job.e.len;
                hi = a.attn.causal ? min(len, pos + 1) : len;
                lo = first_seen(a, pos);
                if (r >= job.t.rows) { lo = job.t.all_lo; hi = job.t.all_hi; }
            }
            float row_m = -INFINITY, row_l = 0.f;
            const float cq = s_cq[job.half][r];
            // The warpgroup's first warp issues its tile's products.
            const bool leads = (warp & 3) == 0;
            const uint32_t it_u = __shfl_sync(0xffffffffu, it, 0);
            auto done = [&](uint32_t one, int which) {
                mma_commit(one, bar + 8 * which);
                if (!job.two && one) mbar_arrive(bar + 8 * which);  // for the tile without rows
            };
            auto await = [&](int which, int s) {  // K or V of step s is converted
                const uint32_t k = it_u + s;
                return bool(__all_sync(0xffffffffu, wait_bar(bar + 8 * (which + k % kStages), (k / kStages) & 1, gone)));
            };
            auto scores = [&](int s) {  // S = Q K^T of step s
                const uint32_t st = (it_u + s) % kStages;
                const uint32_t one = elect_one();
                issue_scores<D>(one, sm, g, st);
                mma_commit(one, bar + 8 * (S_FULL + g));
                done(one, K_EMPTY + st);
                if (one) mbar_arrive(bar + 8 * (S_FULL + g));
            };
            auto values = [&](int s) {  // O += P V of step s
                const uint32_t st = (it_u + s) % kStages;
                const uint32_t one = elect_one();
                issue_values<D>(one, sm, g, st, s > 0);
                mma_commit(one, bar + 8 * (PV_DONE + g));
                done(one, V_EMPTY + st);
            };
            if (leads && await(K_FULL, 0)) {
                tmem_fence_after();
                scores(0);
            }
            bool ok = true;
            int s = 0;
            for (; s < n; ++s) {
                const uint32_t ph = (it_g + s) & 1;
                ok = __all_sync(0xffffffffu, wait_bar(bar + 8 * (S_FULL + g), ph, gone));
                if (!ok) break;
                tmem_fence_after();
                const Places &pl = places[(it + s) % kPlaces];
                const bool whole = !(pl.partial[0] | pl.partial[1] | pl.partial[2] | pl.partial[3]);
                // The step's 128 scores of the row stay in registers; x = score * f + b by groups.  Steps that
                // every row sees whole have code of their own: with the masks' code for all, 512 tokens on
                // 31,232 took 440 us instead of 240 (in an earlier form of this loop).
                auto weights = [&](auto whole_c) -> bool {
                    constexpr bool kWhole = decltype(whole_c)::value;
                    uint32_t x0[32], x1[32], x2[32], x3[32];
                    auto hide = [&](uint32_t (&x)[32], int gi) {  // scores of groups gi, gi + 1 that the row does not see
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int first = max(lo - pl.t0[gi + y], 0), past = min(hi - pl.t0[gi + y], pl.nv[gi + y]);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (e < first || e >= past) x[16 * y + e] = 0xff800000u;  // -infinity
                        }
                    };
                    // f and b of the groups; a group the row does not see at all gets harmless ones, as its
                    // page's scales may be anything
                    float f[kGroups], b[kGroups], iv[4];
#pragma unroll
                    for (int y = 0; y < kGroups; y += 4) {
                        const float4 k4 = *reinterpret_cast<const float4 *>(pl.ks + y), l4 = *reinterpret_cast<const float4 *>(pl.lvs + y);
                        f[y] = k4.x * cq; f[y + 1] = k4.y * cq; f[y + 2] = k4.z * cq; f[y + 3] = k4.w * cq;
                        b[y] = l4.x; b[y + 1] = l4.y; b[y + 2] = l4.z; b[y + 3] = l4.w;
                    }
                    auto unseen = [&](int y) { return min(hi - pl.t0[y], pl.nv[y]) <= max(lo - pl.t0[y], 0); };
                    if constexpr (!kWhole) {
#pragma unroll
                        for (int y = 0; y < kGroups; ++y) {
                            f[y] = f[y] < 1e-37f ? 1e-37f : f[y];  // keeps -infinity * f from being a NaN
                            if (unseen(y)) { f[y] = 1.f; b[y] = 0.f; }
                        }
                    }
                    auto inverses = [&](int y) {  // 1 / scale of groups y .. y + 3
                        const float4 i4 = *reinterpret_cast<const float4 *>(pl.ivs + y);
                        iv[0] = i4.x; iv[1] = i4.y; iv[2] = i4.z; iv[3] = i4.w;
                        if constexpr (!kWhole) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if (unseen(y + x)) iv[x] = 0.f;
                        }
                    };
                    float big = -INFINITY;
                    auto largest = [&](const uint32_t (&x)[32], float f0, float b0, float f1, float b1) {
                        float top[2];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float u = __uint_as_float(x[16 * y]), v = __uint_as_float(x[16 * y + 1]);
#pragma unroll
                            for (int e = 2; e < 14; e += 4) {
                                u = max3(u, __uint_as_float(x[16 * y + e]), __uint_as_float(x[16 * y + e + 1]));
                                v = max3(v, __uint_as_float(x[16 * y + e + 2]), __uint_as_float(x[16 * y + e + 3]));
                            }
                            u = max3(u, __uint_as_float(x[16 * y + 14]), __uint_as_float(x[16 * y + 15]));
                            top[y] = fmaxf(u, v);
                        }
                        // scales are not negative: a group's largest x comes from its largest score
                        big = max3(big, fmaf(top[0], f0, b0), fmaf(top[1], f1, b1));
                    };
                    tmem_ld32(ts, x0);
                    tmem_ld32(ts + 32, x1);
                    tmem_wait_ld();
                    tmem_ld32(ts + 64, x2);
                    tmem_ld32(ts + 96, x3);
                    if constexpr (!kWhole) { hide(x0, 0); hide(x1, 2); }
                    largest(x0, f[0], b[0], f[1], b[1]);
                    largest(x1, f[2], b[2], f[3], b[3]);
                    tmem_wait_ld();
                    if constexpr (!kWhole) { hide(x2, 4); hide(x3, 6); }
                    largest(x2, f[4], b[4], f[5], b[5]);
                    largest(x3, f[6], b[6], f[7], b[7]);
                    inverses(0);
                    const bool grow = big > row_m + kSlack || (row_m == -INFINITY && big > -INFINITY);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float m = grow ? big + kHead : row_m;
                        const float f = grow ? exp2_of(row_m - m) : 1.f;  // 0 from a first maximum
                        row_l *= f;
                        row_m = m;
                        if (s > 0) {
                            if (!__all_sync(0xffffffffu, wait_bar(bar + 8 * (PV_DONE + g), ph ^ 1, gone))) return false;
                            tmem_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) {  // 8 at a time: the scores stay in their registers
                                uint32_t x[8];
                                tmem_ld8(to + 8 * c, x);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                                tmem_st8(to + 8 * c, x);
                            }
                        }
                    }
                    const float ref = row_m == -INFINITY ? 0.f : row_m;
                    auto weigh = [&](const uint32_t (&x)[32], int c, float f0, float b0, float i0, float f1, float b1, float i1) {
                        uint32_t p[16];
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint64_t ff = y ? pair_of(f1, f1) : pair_of(f0, f0), bb = y ? pair_of(b1, b1) : pair_of(b0, b0);
                            uint64_t s0 = 0, s1 = 0;  // two pairs of partial sums
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                float2 u = split_pair(fma_pair(pair_of(__uint_as_float(x[16 * y + e]), __uint_as_float(x[16 * y + e + 1])), ff, bb));
                                float2 v = split_pair(fma_pair(pair_of(__uint_as_float(x[16 * y + e + 2]), __uint_as_float(x[16 * y + e + 3])), ff, bb));
                                u.x = exp2_of(u.x); u.y = exp2_of(u.y); v.x = exp2_of(v.x); v.y = exp2_of(v.y);
                                s0 = add_pair(s0, pair_of(u.x, u.y));
                                s1 = add_pair(s1, pair_of(v.x, v.y));
                                p[8 * y + e / 2] = pack2<KVL_TYPE_HALF>(u.x, u.y);
                                p[8 * y + e / 2 + 1] = pack2<KVL_TYPE_HALF>(v.x, v.y);
                            }
                            const float2 sum = split_pair(add_pair(s0, s1));
                            row_l = fmaf(sum.x + sum.y, y ? i1 : i0, row_l);
                        }
                        tmem_st16(ts + 16 * c, p);
                    };
#pragma unroll
                    for (int y = 0; y < kGroups; ++y) b[y] -= ref;
                    weigh(x0, 0, f[0], b[0], iv[0], f[1], b[1], iv[1]);
                    const float iv2 = iv[2], iv3 = iv[3];
                    inverses(4);
                    weigh(x1, 1, f[2], b[2], iv2, f[3], b[3], iv3);
                    weigh(x2, 2, f[4], b[4], iv[0], f[5], b[5], iv[1]);
                    weigh(x3, 3, f[6], b[6], iv[2], f[7], b[7], iv[3]);
                    return true;
                };
                ok = whole ? weights(std::true_type{}) : weights(std::false_type{});
                if (!ok) break;
                tmem_wait_st();
                tmem_fence_before();
                if (!leads) {
                    meet.arrive<128>(weights_bar(g, ph));
                    continue;
                }
                const bool more = s + 1 < n;
                if (!(ok = await(V_FULL, s) && (!more || await(K_FULL, s + 1)))) break;
                meet.wait<128>(weights_bar(g, ph));
                // The tiles take turns: a tile's two products run one after the other, not mixed with the
                // other tile's, so one tile is at its softmax while the other is at its products.
                if (job.two && (g == 1 || s > 0)) meet.wait<64>(turn_bar(g));
                tmem_fence_after();
                values(s);
                if (more) scores(s + 1);
                if (job.two && (g == 0 || more)) meet.arrive<64>(turn_bar(1 - g));
            }
            if (!ok) leave_steps(meet, leads, job.two, g, it_g, s, n);
            if (ok) {
                ok = __all_sync(0xffffffffu, wait_bar(bar + 8 * (PV_DONE + g), (it_g + n - 1) & 1, gone));
                tmem_fence_after();
            }
            // ---- the row's result, or its part
            const bool complete = job.complete;
            const int rows = job.t.rows, h = job.h;
            const Entry e_ = job.e;
            uint32_t nan_at[D / 32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) nan_at[c] = 0;
            if (ok && CODE == KVL_CODE_FLOAT && *const_cast<volatile int *>(&s_nan) && r < rows) {
                // elements that a NaN code of a seen token reaches, from the steps that were cleared
                for (int gi = job.t.g0 + job.sa * kGroups; gi < min(job.t.g1, job.t.g0 + (job.sa + n) * kGroups); ++gi) {
                    const int blk = gi / per_block, slot = (gi - blk * per_block) * kGroup, t0 = blk * B + slot;
                    const int nv = min(min(kGroup, B - slot), e_.len - t0);
                    const int32_t page = e_.table[blk];
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
            const uint32_t row = job.row_base + r, tok = row / uint32_t(G);
            const int64_t out_row = e_.row0 + tok;
            const int head = h * G + int(row - tok * G);
            const float inv = row_l == 0.f ? 0.f : 1.f / row_l;
            float *part = a.parts + (int64_t(blockIdx.x) * 2 + (job.sa == 0 ? 1 : 0)) * C::kPartFloats;
            uint8_t *dst = static_cast<uint8_t *>(a.attn.out.data) + out_row * a.attn.out.row_stride + head * a.attn.out.head_stride;
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
                    if (r < rows) {
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
                if (r < rows) {
                    if (!complete) {
                        part[r] = row_m;
                        part[kJobRows + r] = row_l;
                    } else if (a.attn.lse) {
                        a.attn.lse[out_row * a.attn.n_heads + head] =
                            row_l == 0.f ? -INFINITY : (row_m + __log2f(row_l)) * (1.f / kLog2e);
                    }
                }
            }
            tmem_fence_before();
        }
        if (job.n > 0 && !job.complete) {
            // parts of this job: shares first .. last; the one that arrives last joins them
            const int first = int(job.cut.share_of(job.u0)), last = int(job.cut.share_of(job.u0 + job.t.steps - 1));
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = arrive_part(a, job, *gone);
            __syncthreads();
            if (s_last) {
                __threadfence();
                const int n_rows = job.t.rows, n_parts = last - first + 1;
                // 32 elements of a row a thread and turn
                for (int x = tid; x < kJobRows * (D / 32); x += kThreads) {
                    const int r = x & (kJobRows - 1), c = x / kJobRows;
                    if (r >= n_rows) continue;
                    auto part_of = [&](int b) { return a.parts + (int64_t(first + b) * 2 + (b == 0)) * C::kPartFloats; };
                    float big = -INFINITY, sum = 0.f;
#pragma unroll 4
                    for (int b = 0; b < n_parts; ++b) big = fmaxf(big, __ldcg(part_of(b) + r));
                    float4 v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                    for (int b = 0; b < n_parts; ++b) {
                        const float *p = part_of(b);
                        const float mb = __ldcg(p + r), lb = __ldcg(p + kJobRows + r);
                        const float f = mb == -INFINITY ? 0.f : exp2_of(mb - big);
                        sum += lb * f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(p + 2 * kJobRows) + int64_t(8 * c + e) * kJobRows + r);
                            v[e].x += y.x * f; v[e].y += y.y * f; v[e].z += y.z * f; v[e].w += y.w * f;
                        }
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const uint32_t row = job.row_base + r, tok = row / uint32_t(G);
                    const int64_t out_row = job.e.row0 + tok;
                    const int head = job.h * G + int(row - tok * G);
                    uint8_t *dst = static_cast<uint8_t *>(a.attn.out.data) + out_row * a.attn.out.row_stride +
                                   head * a.attn.out.head_stride + 64 * c;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w[8] = {v[2 * e].x * inv, v[2 * e].y * inv, v[2 * e].z * inv, v[2 * e].w * inv,
                                            v[2 * e + 1].x * inv, v[2 * e + 1].y * inv, v[2 * e + 1].z * inv, v[2 * e + 1].w * inv};
                        if (32 * c + 8 * e < d) store8<TYPE>(dst + 16 * e, w);
                    }
                    if (a.attn.lse && c == 0)
                        a.attn.lse[out_row * a.attn.n_heads + head] =
                            sum == 0.f ? -INFINITY : (big + __log2f(sum)) * (1.f / kLog2e);
                }
            }
        }
        __syncthreads();  // tensor memory is free again, the next job's Q in its place
        tmem_fence_after();
        if (tid == 0) {
            job = next;
            s_nan = 0;
        }
        __syncthreads();
        if (*gone || job.n == 0) break;
    }
    if (*gone) {
        if (tid == 0) report(a.report, KVL_ETIMEOUT, blockIdx.x);
        if (warp == 8) arrive_without_result(a, job, lane);
        // let the products in flight end (bounded) before their memory goes, one issuing thread's after
        // the other's
        if (warp == 0) {
            mma_commit(elect_one(), bar + 8 * LEAVE);
            mbar_wait_bounded(bar + 8 * LEAVE, 0);
        }
        __syncthreads();
        if (warp == 4) {
            mma_commit(elect_one(), bar + 8 * LEAVE);
            mbar_wait_bounded(bar + 8 * LEAVE, 1);
        }
    }
    __syncthreads();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
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

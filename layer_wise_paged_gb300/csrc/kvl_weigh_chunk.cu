// kvl_weigh_chunk.cu -- the weight that many rows a sequence give each cached token: prompts, and the last rows of
// one that judge it.
//
// 2 d operations and one exponential for each (row, token), and no value product after it, so there is no chain:
// S^T = K Q^T with tokens in the 128-high operand puts a token into each thread's lane of tensor memory, whose
// weights it adds up in registers; nothing goes back.  A CTA holds 256 tokens (two halves of 128) of one KV head
// after another as halves in shared memory, and the rows stream past them 128 at a time, already scaled, converted
// and swizzled by a first kernel, as one bulk copy a step (so a step reads 33 KB for 256 x 128 scores).
//   warps 0-15       weights: a thread a token of each half and a quarter of a step's rows, so that what is read of a row
//                    from shared memory, which the products keep busy half of the time, serves two tokens
//   warps 16-19      read the K codes of the next head from the pages, convert them to halves (exact)
//   warp 20          issues the products: two of 128 x 128 a step, into two sets of accumulators in turn
//   warp 21          brings the rows
// Work: (entry, 256 tokens) is a job of (KV heads x row chunks that see it) steps; the steps of all jobs in a row
// are cut into equal contiguous shares, one a CTA.  A job that crosses shares leaves its sums in the workspace, and
// the CTA that arrives last adds them up in the order of the shares.
//
// Every wait is bounded: past the limit a flag is raised, every role leaves, and the report says KVL_ETIMEOUT.
#include "kvl_tcgen.cuh"
#include "kvl_weigh.cuh"

namespace kvl {
namespace {

constexpr int kWeighing = 16;                 // warps
constexpr int kWarps = kWeighing + 6;
constexpr int kThreads = kWarps * 32;
constexpr int kTokens = 256;                  // of a job
constexpr int kJobGroups = kTokens / kGroup;  // 16
constexpr int kRows = 128;                    // of a step
constexpr int kScales = 4;                    // heads whose scales are kept: the weights of a step may be two heads
                                              // behind the conversion, which is one ahead of its own
constexpr int kConsts = 8;                    // steps whose rows' factors are kept: two ahead of the products, and two
                                              // behind whose weights may still read theirs (they give a step's
                                              // accumulators back before they have used all of it)
constexpr int kConstBytes = kRows * 4 + 16;
constexpr int kBatch = 512;                   // entries whose steps are held at a time

template <int D>
struct Chunk {
    static constexpr int kHalfBytes = 128 * D * 2;      // 128 tokens of K, or a step's rows
    static constexpr int kK = 0;                        // [2][2 halves]
    static constexpr int kQ = 4 * kHalfBytes;           // [2]
    static constexpr int kSmem = kQ + 2 * kHalfBytes + 1024;
    static constexpr int kTileBytes = kHalfBytes + kConstBytes;  // of the workspace: rows, their factors and offsets
};

enum Bar { K_FULL = 0, K_EMPTY = 2, Q_FULL = 4, Q_EMPTY = 6, S_FULL = 8, S_EMPTY = 10, JOIN = 12, SUM_FULL = 13, SUM_EMPTY = 14, LEAVE = 15, BARS = 16 };

// Workspace: [counters of the shares][parts: two a share, 256 sums][row tiles: rows, their
// offsets, their factor, negative where a row among them gives nothing].  Tile of entry i's chunk c: number
// row0 * G / 128 + i + c, of which no two entries' meet.
__host__ __device__ constexpr size_t counter_bytes(int sms) { return size_t(sms) * 4 + 255 & ~size_t(255); }
__host__ __device__ constexpr size_t part_bytes(int sms) { return size_t(sms) * 2 * kTokens * 4; }

struct ChunkArgs {
    WeighArgs w;
    uint32_t *counters;
    float *parts;
    uint8_t *tiles;
    int32_t sms;
};

// ---- rows: as halves, in the layout the products read.  A tile's rows are scaled by one power of two, which takes
// their largest element into [2^14, 2^15): one factor for all.  What is lost is below 2^-39 of that element. ------------

__device__ __forceinline__ int find_entry_of_tile(const kvl_sequences &s, int G, int64_t id, int lane)
{
    int lo = 0, hi = s.n_seq;  // the last i with starts[i] G / 128 + i <= id is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool below = i < hi && int64_t(max(s.starts[i], 0)) * G / kRows + i <= id;
        const unsigned m = __ballot_sync(0xffffffffu, below);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

template <int TYPE, int D>
__global__ void __launch_bounds__(256) weigh_rows_prepare_kernel(const __grid_constant__ ChunkArgs a)
{
    const AttendArgs &t = a.w.t;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    allow_dependents_launch();
    const int H = t.cache.n_kv_heads, G = t.attn.n_heads / H, d = t.cache.head_dim, h = blockIdx.y;
    if (blockIdx.x == 0 && h == 0)
        for (int x = threadIdx.x; x < a.sms; x += 256) a.counters[x] = 0;
    const int i = find_entry_of_tile(t.seqs, G, blockIdx.x, lane);
    const Entry e = load_entry(t.seqs, t.cache.block_tokens, i, nullptr);
    const int64_t chunk = int64_t(blockIdx.x) - (int64_t(e.row0) * G / kRows + i), rows = int64_t(e.fresh) * G;
    if (chunk < 0 || chunk * kRows >= rows) return;
    uint8_t *tile = a.tiles + (int64_t(blockIdx.x) * H + h) * Chunk<D>::kTileBytes;
    float *consts = reinterpret_cast<float *>(tile + Chunk<D>::kHalfBytes);
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a warp's vector
    constexpr int kTurns = kRows / (8 * kPer);
    __shared__ float s_most[8];
    const int at = (lane % kLanes) * 8;
    uint4 raw[kTurns];
    bool infinite = false;
    float z_of[kTurns], amax = 0.f;  // of finite elements
#pragma unroll
    for (int x = 0; x < kTurns; ++x) {
        const int64_t row = chunk * kRows + (warp + 8 * x) * kPer + lane / kLanes;
        raw[x] = make_uint4(0, 0, 0, 0);
        z_of[x] = 0.f;
        if (row < rows && at < d) {
            const int tok = int(row / G), head = h * G + int(row - int64_t(tok) * G);
            z_of[x] = a.w.lse[(int64_t(e.row0) + tok) * t.attn.n_heads + head];
            raw[x] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(t.attn.q.data) +
                                                      (int64_t(e.row0) + tok) * t.attn.q.row_stride + int64_t(head) * t.attn.q.head_stride + 2 * at);
        }
    }
#pragma unroll
    for (int x = 0; x < kTurns; ++x) {
        float v[8];
        if (isinf(z_of[x])) {  // gives nothing, whatever it holds
            raw[x] = make_uint4(0, 0, 0, 0);
            infinite = true;
        }
        load8<TYPE>(reinterpret_cast<const uint8_t *>(&raw[x]), v);
#pragma unroll
        for (int y = 0; y < 8; ++y) amax = fmaxf(amax, isfinite(v[y]) ? fabsf(v[y]) : 0.f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_most[warp] = amax;
    // (rows that are not there need no mark: a NaN key that all others see counts, or all of them are marked)
    const bool nothing = __syncthreads_or(infinite);
#pragma unroll
    for (int x = 0; x < 8; ++x) amax = fmaxf(amax, s_most[x]);
    // 2^e <= amax < 2^(e + 1), e held to what leaves both factors normal
    const int ex = max(-100, int(__float_as_uint(amax) >> 23) - 127);
    const float up = __uint_as_float(uint32_t(14 - ex + 127) << 23), down = __uint_as_float(uint32_t(ex - 14 + 127) << 23);
#pragma unroll
    for (int x = 0; x < kTurns; ++x) {
        const int r = (warp + 8 * x) * kPer + lane / kLanes;
        float v[8];
        load8<TYPE>(reinterpret_cast<const uint8_t *>(&raw[x]), v);
        uint4 p;
        p.x = pack2<KVL_TYPE_HALF>(v[0] * up, v[1] * up);
        p.y = pack2<KVL_TYPE_HALF>(v[2] * up, v[3] * up);
        p.z = pack2<KVL_TYPE_HALF>(v[4] * up, v[5] * up);
        p.w = pack2<KVL_TYPE_HALF>(v[6] * up, v[7] * up);
        const int unit = at / 8;
        *reinterpret_cast<uint4 *>(tile + (unit >> 3) * (kRows * 128) + r * 128 + (((unit & 7) ^ (r & 7)) << 4)) = p;
    }
    if (threadIdx.x < kRows) {
        // a row that is not there, or whose lse is infinite, gives nothing: an offset of -infinity
        const int64_t row = chunk * kRows + threadIdx.x;
        float z = INFINITY;
        if (row < rows) {
            const int tok = int(row / G), head = h * G + int(row - int64_t(tok) * G);
            z = a.w.lse[(int64_t(e.row0) + tok) * t.attn.n_heads + head];
        }
        consts[threadIdx.x] = isinf(z) ? -INFINITY : -z * kLog2e;
    }
    if (threadIdx.x == 0) consts[kRows] = t.attn.sm_scale * kLog2e * (nothing ? -down : down);
}

// ---- work ---------------------------------------------------------------------------------------------------

// An entry's tokens that some row sees, as tiles of 256 slots.
struct Span {
    Entry e;
    int32_t g0, groups, tiles, chunks;
};

__device__ __forceinline__ Span span_of(const WeighArgs &w, int i, void *rep)
{
    const AttendArgs &a = w.t;
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup;
    Span s;
    s.e = load_entry(a.seqs, B, i, rep);
    if (s.e.len > w.tokens) {
        report(rep, KVL_ERANGE, i);
        s.e.len = s.e.fresh = 0;
    }
    s.g0 = group_of(first_seen(a, s.e.len - s.e.fresh), B, per_block);
    s.groups = s.e.fresh > 0 && s.e.len > 0 ? group_of(s.e.len - 1, B, per_block) + 1 - s.g0 : 0;
    s.tiles = (s.groups + kJobGroups - 1) / kJobGroups;
    s.chunks = int32_t((int64_t(s.e.fresh) * (a.attn.n_heads / a.cache.n_kv_heads) + kRows - 1) / kRows);
    return s;
}

// The first token of an entry's group g (a group past the end: the end, or more).
__device__ __forceinline__ int32_t token_of(const Span &s, int32_t g, int32_t B, int32_t per_block)
{
    const int32_t blk = (s.g0 + g) / per_block;
    return blk * B + (s.g0 + g - blk * per_block) * kGroup;
}

// Row chunks [ca, ca + n) see tokens of tile t; at least one is walked, so that the tile's masses are written.
__device__ __forceinline__ void chunks_of(const WeighArgs &w, const Span &s, int t, int32_t &ca, int32_t &n)
{
    const AttendArgs &a = w.t;
    const int B = a.cache.block_tokens, per_block = (B + kGroup - 1) / kGroup, G = a.attn.n_heads / a.cache.n_kv_heads;
    const int32_t pos0 = s.e.len - s.e.fresh;
    int64_t first = 0, past = s.chunks;
    if (a.attn.causal) {
        const int64_t row = (int64_t(token_of(s, t * kJobGroups, B, per_block)) - pos0) * G;
        if (row > 0) first = row / kRows;
    }
    if (a.attn.window > 0) {
        const int64_t end = min(s.e.len, token_of(s, min((t + 1) * kJobGroups, s.groups), B, per_block));
        past = min(past, ((end - 1 + a.attn.window - pos0) * G + kRows - 1) / kRows);
    }
    first = min(first, int64_t(s.chunks - 1));
    ca = int32_t(first);
    n = int32_t(max(past - first, int64_t(1)));
}

// Steps of an entry; a warp's lanes take a tile each.
__device__ __forceinline__ uint64_t warp_steps(const WeighArgs &w, const Span &s, int lane)
{
    uint64_t sum = 0;
    for (int t = lane; t < s.tiles; t += 32) {
        int32_t ca, n;
        chunks_of(w, s, t, ca, n);
        sum += uint64_t(w.t.cache.n_kv_heads) * n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// A walk over the jobs of a share, each role's own.
struct Walk {
    uint32_t u, u_end;
    int32_t entry, tile;
    Span s;
    int32_t ca, n;      // the job's chunks
    int32_t x0, taken;  // its steps in this share: step x is KV head x / n, chunk ca + x % n
    uint32_t u0;        // the unit of its first step

    // where off steps of entry i precede unit u; by one whole warp
    __device__ __forceinline__ void begin(const WeighArgs &w, uint32_t first, uint32_t end, int i, uint32_t off, int lane)
    {
        u = first;
        u_end = end;
        entry = i;
        s = span_of(w, i, nullptr);
        const int H = w.t.cache.n_kv_heads;
        tile = 0;
        for (int base = 0; base < s.tiles; base += 32) {
            int32_t c = 0, m = 0;
            if (base + lane < s.tiles) chunks_of(w, s, base + lane, c, m);
            uint32_t sum = uint32_t(m) * H, mine = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, off < sum);
            if (past) {
                const int l = __ffs(past) - 1;
                tile = base + l;
                off -= __shfl_sync(0xffffffffu, sum - mine, l);
                break;
            }
            off -= __shfl_sync(0xffffffffu, sum, 31);
        }
        here(w, off);
    }
    __device__ __forceinline__ void here(const WeighArgs &w, uint32_t off)
    {
        chunks_of(w, s, tile, ca, n);
        x0 = int32_t(off);
        u0 = u - off;
        taken = int32_t(min(uint32_t(n) * w.t.cache.n_kv_heads - off, u_end - u));
    }
    __device__ __forceinline__ bool next(const WeighArgs &w)
    {
        u += taken;
        if (u >= u_end) return false;
        if (++tile >= s.tiles) {
            tile = 0;
            do s = span_of(w, ++entry, nullptr); while (s.tiles == 0);
        }
        here(w, 0);
        return true;
    }
    __device__ __forceinline__ bool complete(const WeighArgs &w) const { return taken == n * w.t.cache.n_kv_heads; }
};

template <int CODE, int D>
__global__ void __launch_bounds__(kThreads, 1) weigh_chunk_kernel(const __grid_constant__ ChunkArgs args)
{
    using C = Chunk<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long bars[BARS];
    __shared__ uint32_t s_units[kBatch];
    __shared__ __align__(16) float s_consts[kConsts][kConstBytes / 4];
    __shared__ float s_scales[kScales][kJobGroups];
    __shared__ float s_sum[3][kTokens];
    __shared__ uint32_t s_off, s_tmem;
    __shared__ int s_entry, s_gone, s_last;
    const WeighArgs &w = args.w;
    const AttendArgs &a = w.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int G = a.attn.n_heads / H, per_block = (B + kGroup - 1) / kGroup;
    const int64_t N = a.cache.pool_blocks, plane = int64_t(a.layer) * 2 * N;

    // ---- this CTA's share: the entries' steps a batch at a time, their sum, then the entry that holds the first
    // (where starts descend two entries' row tiles may have one number: nothing is weighed)
    uint64_t before = 0;
    uint32_t u = 0;
    bool falls = false;
    Cut cut;
    for (int pass = 0; pass < 2; ++pass) {
        for (int base = 0; base < a.seqs.n_seq; base += kBatch) {
            const int n = min(kBatch, a.seqs.n_seq - base);
            if (pass == 0 || a.seqs.n_seq > kBatch) {
                __syncthreads();
                for (int i = warp; i < n; i += kWarps) {
                    const Span s = span_of(w, base + i, pass == 0 && blockIdx.x == 0 && lane == 0 ? a.report : nullptr);
                    const uint64_t steps = warp_steps(w, s, lane);
                    falls = falls || a.seqs.starts[base + i + 1] < a.seqs.starts[base + i];
                    if (lane == 0) s_units[i] = uint32_t(min(steps, kMostUnits));
                }
                falls = __syncthreads_or(falls);
            }
            for (int i = 0; i < n; i += 32) {
                uint64_t x = i + lane < n ? s_units[i + lane] : 0, sum = x;
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
                            s_entry = base + i + l;
                            s_off = u - at;
                        }
                        base = a.seqs.n_seq;  // found: leave both loops
                        break;
                    }
                }
                before += __shfl_sync(0xffffffffu, sum, 31);
            }
        }
        if (pass == 0) {
            if (before == 0 || before >= kMostUnits || falls) {
                if (before >= kMostUnits && blockIdx.x == 0 && tid == 0) report(a.report, KVL_ERANGE, a.seqs.n_seq);
                grid_dependency_wait();  // the rows' kernel has ended when this one has
                return;
            }
            cut = Cut(uint32_t(before), min(gridDim.x, uint32_t(before)));
            if (blockIdx.x >= cut.shares) {
                grid_dependency_wait();
                return;
            }
            u = cut.start(blockIdx.x);
            before = 0;
        }
    }

    const uint32_t bar = smem_u32(bars);
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sm = smem_u32(smem);
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar + 8 * (K_FULL + x), 4);   // the converting warps
            mbar_init(bar + 8 * (K_EMPTY + x), 1);  // the head's last product
            mbar_init(bar + 8 * (Q_FULL + x), 1);   // the bringing thread, and its bytes
            mbar_init(bar + 8 * (Q_EMPTY + x), 1);  // the step's products
            mbar_init(bar + 8 * (S_FULL + x), 2);   // the step's products, and the issuing thread, by which K's scales
                                                    // and the rows' factors reach the weighing warps
            mbar_init(bar + 8 * (S_EMPTY + x), kWeighing);
        }
        mbar_init(bar + 8 * JOIN, 4);        // the first side's warps
        mbar_init(bar + 8 * SUM_FULL, 12);   // the other sides' sums of a job; the first side has them
        mbar_init(bar + 8 * SUM_EMPTY, 4);
        mbar_init(bar + 8 * LEAVE, 1);
        fence_mbar_init();
        s_gone = 0;
    }
    if (warp == kWeighing + 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem;  // columns: two sets of two halves of 128
    volatile int *gone = &s_gone;
    auto wait = [&](int which, uint32_t parity) {  // by whole warps, whose lanes go on or give up together
        return bool(__all_sync(0xffffffffu, wait_bar(bar + 8 * which, parity, gone)));
    };
    Walk job;
    job.begin(w, u, cut.start(blockIdx.x + 1), s_entry, s_off, lane);

    if (warp < kWeighing) {
        // ---- weights: tokens slot and slot + 128 of the job, rows 32 side .. of every step
        const int side = warp >> 2, slot = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (uint32_t(warp & 3) << 21) + side * 32;
        uint32_t s = 0, k = 0, joins = 0, sums = 0;  // steps, heads, joins and jobs so far
        bool ok = true;
        do {
            const int pos0 = job.s.e.len - job.s.e.fresh, rows = job.s.e.fresh * G;  // (at most 2^26)
            const int sq = a.seqs.slots ? a.seqs.slots[job.entry] : job.entry;
            const float *in = w.mass_in + int64_t(sq) * w.in_stride;
            float *out = w.mass_out + int64_t(sq) * w.out_stride;
            int token[2];  // -1: none
            float held[2], sum[2] = {0.f, 0.f};
            int32_t page[2];
            // rows [see_a, see_b) of the entry see the token; a lane without one may see any
            int see_a[2], see_b[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int g = job.tile * kJobGroups + (slot + 128 * y) / kGroup;
                const int blk = (job.s.g0 + g) / per_block, at = (job.s.g0 + g - blk * per_block) * kGroup + slot % kGroup;
                const int j = blk * B + at;
                const bool there = g < job.s.groups && at < B && j < job.s.e.len;
                token[y] = there ? j : -1;
                // (both on their way during the steps)
                held[y] = side || !there || (w.begin && j >= pos0) ? 0.f : in[j];
                page[y] = there && !side ? job.s.e.table[blk] : -1;
                see_a[y] = there && a.attn.causal ? int(max((int64_t(j) - pos0) * G, int64_t(0))) : 0;  // (past the rows, if none)
                see_b[y] = there && a.attn.window > 0 ? int(max(min((int64_t(j) + a.attn.window - pos0) * G, int64_t(rows)), int64_t(0))) : rows;
            }
            // (of most tiles every row sees every token)
            const bool always = __all_sync(0xffffffffu, see_a[0] == 0 && see_a[1] == 0 && see_b[0] >= rows && see_b[1] >= rows);
            int c = job.x0 % job.n;
            for (int x = 0; x < job.taken; ++x, ++s) {
                const uint32_t set = s & 1, ph = (s >> 1) & 1;
                ok = wait(S_FULL + set, ph);
                if (!ok) break;
                tmem_fence_after();
                const int row_a = (job.ca + c) * kRows + 32 * side, n_rows = min(32, rows - row_a);
                const float *consts = s_consts[s % kConsts] + side * 32;
                const uint32_t ts = lanes + set * 256;
                if (n_rows > 0) {
                    const float f = consts[kRows - side * 32];
                    float kf[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) kf[y] = s_scales[k % kScales][(slot + 128 * y) / kGroup] * fabsf(f);
                    int from[2] = {0, 0}, to[2] = {kRows, kRows};
                    // by some lane's row; by all, all of which count: one of an infinite lse gives nothing even of a NaN
                    // key, whose product is a NaN whatever the row
                    bool seen[2] = {true, true}, whole = f > 0.f;
                    if (!always) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            from[y] = see_a[y] - row_a;
                            to[y] = see_b[y] - row_a;
                            seen[y] = __any_sync(0xffffffffu, from[y] < n_rows && to[y] > 0);
                            whole = whole && from[y] <= 0 && to[y] >= n_rows;
                        }
                        whole = __all_sync(0xffffffffu, whole);
                    }
                    const uint64_t kk[2] = {pair_of(kf[0], kf[0]), pair_of(kf[1], kf[1])};
                    uint64_t add[2][2] = {{0, 0}, {0, 0}};
                    uint32_t v[2][16];
#pragma unroll
                    for (int col = 0; col < 32; col += 16) {
                        tmem_ld16(ts + col, v[0]);
                        tmem_ld16(ts + col + 128, v[1]);
                        tmem_wait_ld();
                        if (col == 16) {
                            tmem_fence_before();
                            if (lane == 0) mbar_arrive(bar + 8 * (S_EMPTY + set));
                        }
                        auto weights = [&](int y, int i, uint64_t b) {  // of rows col + i, col + i + 1
                            float2 q = split_pair(fma_pair(pair_of(__uint_as_float(v[y][i]), __uint_as_float(v[y][i + 1])), kk[y], b));
                            return make_float2(exp2_of(q.x), exp2_of(q.y));
                        };
                        if (whole) {
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                const float4 b = *reinterpret_cast<const float4 *>(consts + col + 4 * p);
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const float2 q = weights(y, 4 * p, pair_of(b.x, b.y)), z = weights(y, 4 * p + 2, pair_of(b.z, b.w));
                                    add[y][0] = add_pair(add[y][0], pair_of(q.x, q.y));
                                    add[y][1] = add_pair(add[y][1], pair_of(z.x, z.y));
                                }
                            }
                        } else {
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                if (!seen[y]) continue;
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    const float2 b = *reinterpret_cast<const float2 *>(consts + col + i);
                                    float2 q = weights(y, i, pair_of(b.x, b.y));
                                    if (col + i < from[y] || col + i >= to[y] || b.x == -INFINITY) q.x = 0.f;
                                    if (col + i + 1 < from[y] || col + i + 1 >= to[y] || b.y == -INFINITY) q.y = 0.f;
                                    add[y][0] = add_pair(add[y][0], pair_of(q.x, q.y));
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 t = split_pair(add_pair(add[y][0], add[y][1]));
                        sum[y] += t.x + t.y;
                    }
                } else if (lane == 0) {
                    mbar_arrive(bar + 8 * (S_EMPTY + set));
                }
                if (++c == job.n) c = 0;
                if (c == 0 || x + 1 == job.taken) ++k;
            }
            if (!ok) break;
            if (side) {
                if (!(ok = wait(SUM_EMPTY, (sums & 1) ^ 1))) break;
                s_sum[side - 1][slot] = sum[0];
                s_sum[side - 1][slot + 128] = sum[1];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * SUM_FULL);
                ++sums;
                // tokens before the first that a row sees
                if (job.tile == 0 && job.x0 == 0 && in != out) {
                    const int past = token_of(job.s, 0, B, per_block);
                    for (int y = slot + 128 * (side - 1); y < past; y += 384) out[y] = in[y];
                }
                continue;
            }
            if (!(ok = wait(SUM_FULL, sums++ & 1))) break;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int z = 0; z < 3; ++z) sum[y] += s_sum[z][slot + 128 * y];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8 * SUM_EMPTY);
            bool last = true;
            if (!job.complete(w)) {
                const uint32_t first = cut.share_of(job.u0), end = cut.share_of(job.u0 + uint32_t(job.n) * H - 1);
                float *part = args.parts + (int64_t(blockIdx.x) * 2 + (job.x0 == 0 ? 1 : 0)) * kTokens + slot;
                part[0] = sum[0];
                part[128] = sum[1];
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * JOIN);
                if (!(ok = wait(JOIN, joins++ & 1))) break;
                if (warp == 0 && lane == 0) {
                    s_last = atomicAdd(&args.counters[first], 1u) == end - first;
                    __threadfence();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * JOIN);
                if (!(ok = wait(JOIN, joins++ & 1))) break;
                last = s_last;
                if (last) {
                    sum[0] = sum[1] = 0.f;
                    for (uint32_t b = first; b <= end; ++b) {
                        const float *p = args.parts + (int64_t(b) * 2 + (b == first ? 1 : 0)) * kTokens + slot;
                        sum[0] += __ldcg(p);
                        sum[1] += __ldcg(p + 128);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (token[y] < 0) continue;
                const bool seen = page[y] >= 0 && page[y] < N;
                if (!seen && slot % kGroup == 0) report(a.report, KVL_ERANGE, job.entry);
                if (last) out[token[y]] = seen ? held[y] + sum[y] : held[y];
            }
        } while (job.next(w));
    } else if (warp < kWeighing + 4) {
        // ---- convert K: warp cw's four groups of the tile, two on their way while another is converted
        const int cw = warp - kWeighing;
        const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
        constexpr int kPer = 512 / D, kVecs = kGroup / kPer;  // rows of a warp's vector, vectors of a group
        // 8 lanes of a shared-memory phase write 4 chunks of an even and of an odd row: with the swizzle, 8
        // different 16-byte columns
        const int ch = (lane & 3) | (D == 128 ? (lane >> 4) << 2 : 0), rw = D == 128 ? (lane >> 2) & 3 : lane >> 2;
        uint32_t k = 0;
        bool ok = true;
        do {
            // lane l looks after the warp's group l: tokens 64 cw + 16 l of the tile
            int32_t page = -1, nv = 0, t0 = 0;
            if (lane < 4) {
                const int g = job.tile * kJobGroups + cw * 4 + lane;
                if (g < job.s.groups) {
                    const int blk = (job.s.g0 + g) / per_block, at = (job.s.g0 + g - blk * per_block) * kGroup;
                    t0 = blk * B + at;
                    nv = min(min(kGroup, B - at), job.s.e.len - t0);
                    page = nv > 0 ? job.s.e.table[blk] : -1;
                    if (page < 0 || page >= N) { page = -1; nv = 0; }
                }
            }
            const int ha = job.x0 / job.n, hb = (job.x0 + job.taken - 1) / job.n;
            uint4 reg[2][kVecs];
            auto fetch = [&](uint4 (&r)[kVecs], int l, int h) {  // group l of head h
                const int32_t pg = __shfl_sync(0xffffffffu, page, l), tt = __shfl_sync(0xffffffffu, t0, l);
                int valid = __shfl_sync(0xffffffffu, nv, l);
                if (ch * 16 >= d) valid = 0;
                const uint8_t *src = codes + (((plane + max(pg, 0)) * B + tt % B) * H + h) * d + ch * 16;
#pragma unroll
                for (int x = 0; x < kVecs; ++x) {
                    r[x] = make_uint4(0, 0, 0, 0);
                    if (x * kPer + rw < valid) r[x] = __ldg(reinterpret_cast<const uint4 *>(src + int64_t(x * kPer + rw) * H * d));
                }
            };
            auto scale = [&](int h) { return page >= 0 ? __ldg(a.cache.scales + (plane + page) * H + h) : 0.f; };
            float sc = scale(ha);
            fetch(reg[0], 0, ha);
            fetch(reg[1], 1, ha);
            for (int h = ha; h <= hb; ++h, ++k) {
                const uint32_t st = k & 1;
                ok = wait(K_EMPTY + st, ((k >> 1) & 1) ^ 1);
                if (!ok) break;
                if (lane < 4) s_scales[k % kScales][cw * 4 + lane] = sc;
                if (h < hb) sc = scale(h + 1);
                uint8_t *dst = smem + C::kK + (st * 2 + (cw >> 1)) * C::kHalfBytes;
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    uint4 (&z)[kVecs] = reg[l & 1];
#pragma unroll
                    for (int x = 0; x < kVecs; ++x) {
                        const int r = (cw & 1) * 64 + l * kGroup + x * kPer + rw;
                        uint4 lo, hi;
                        codes_of<CODE>(z[x].x, lo.x, lo.y);
                        codes_of<CODE>(z[x].y, lo.z, lo.w);
                        codes_of<CODE>(z[x].z, hi.x, hi.y);
                        codes_of<CODE>(z[x].w, hi.z, hi.w);
                        uint8_t *p = dst + (ch >> 2) * (128 * 128) + r * 128;
                        const int un = (ch & 3) * 2;
                        *reinterpret_cast<uint4 *>(p + ((un ^ (r & 7)) << 4)) = lo;
                        *reinterpret_cast<uint4 *>(p + (((un + 1) ^ (r & 7)) << 4)) = hi;
                    }
                    if (l < 2 || h < hb) fetch(z, (l + 2) & 3, l < 2 ? h : h + 1);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar + 8 * (K_FULL + st));
            }
        } while (ok && job.next(w));
    } else if (warp == kWeighing + 4) {
        // ---- products
        uint32_t s = 0, k = 0;
        bool ok = true;
        do {
            const int rows = job.s.e.fresh * G;
            int c = job.x0 % job.n;
            for (int x = 0; x < job.taken; ++x, ++s) {
                const uint32_t st = s & 1, ph = (s >> 1) & 1, kst = k & 1;
                if ((x == 0 || c == 0) && !(ok = wait(K_FULL + kst, (k >> 1) & 1))) break;
                if (!(ok = wait(Q_FULL + st, ph) && wait(S_EMPTY + st, ph ^ 1))) break;
                tmem_fence_after();
                const int n_rows = min(kRows, rows - (job.ca + c) * kRows), cols = (n_rows + 31) / 32 * 32;
                const bool last = c + 1 == job.n || x + 1 == job.taken;
                const uint32_t one = elect_one();
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint64_t kd = matrix_desc(sm + C::kK + (kst * 2 + half) * C::kHalfBytes, 16, 1024);
                    uint64_t qd = matrix_desc(sm + C::kQ + st * C::kHalfBytes, 16, 1024);
#pragma unroll 1
                    for (int y = 0; y < D / 64; ++y) {
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            mma_smem(one, tmem + st * 256 + half * 128, kd + 2 * z, qd + 2 * z, instr_desc(cols, false), y + z > 0);
                        kd += 128 * 128 >> 4;
                        qd += 128 * 128 >> 4;
                    }
                }
                mma_commit(one, bar + 8 * (S_FULL + st));
                mma_commit(one, bar + 8 * (Q_EMPTY + st));
                if (last) mma_commit(one, bar + 8 * (K_EMPTY + kst));
                if (one) mbar_arrive(bar + 8 * (S_FULL + st));
                __syncwarp();
                if (++c == job.n) c = 0;
                if (last) ++k;
            }
        } while (ok && job.next(w));
        // the products in flight end (bounded) before their memory goes
        if (ok && k > 0) ok = wait(K_EMPTY + ((k - 1) & 1), ((k - 1) >> 1) & 1);
        if (!ok) {
            mma_commit(elect_one(), bar + 8 * LEAVE);
            mbar_wait_bounded(bar + 8 * LEAVE, 0);
        }
    } else {
        // ---- rows.  (Only these, and the counters of joins, which come after them, are the first kernel's.)
        grid_dependency_wait();
        uint32_t s = 0;
        bool ok = true;
        do {
            const int64_t first = int64_t(job.s.e.row0) * G / kRows + job.entry + job.ca;
            int c = job.x0 % job.n, h = job.x0 / job.n;
            for (int x = 0; x < job.taken; ++x, ++s) {
                const uint32_t st = s & 1, ph = (s >> 1) & 1;
                if (!(ok = wait(Q_EMPTY + st, ph ^ 1))) break;
                if (lane == 0) {
                    const uint8_t *tile = args.tiles + ((first + c) * H + h) * C::kTileBytes;
                    mbar_arrive_expect_tx(bar + 8 * (Q_FULL + st), C::kTileBytes);
                    bulk_load(sm + C::kQ + st * C::kHalfBytes, tile, C::kHalfBytes, bar + 8 * (Q_FULL + st));
                    bulk_load(smem_u32(s_consts[s % kConsts]), tile + C::kHalfBytes, kConstBytes, bar + 8 * (Q_FULL + st));
                }
                __syncwarp();
                if (++c == job.n) {
                    c = 0;
                    ++h;
                }
            }
        } while (ok && job.next(w));
        // copies in flight end (bounded) before their memory goes
        for (uint32_t x = s > 2 ? s - 2 : 0; x < s; ++x) mbar_wait_bounded(bar + 8 * (Q_FULL + (x & 1)), (x >> 1) & 1);
    }
    __syncthreads();
    if (*gone && tid == 0) report(a.report, KVL_ETIMEOUT, blockIdx.x);
    grid_dependency_wait();
    if (warp == kWeighing + 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int CODE, int TYPE, int D>
kvl_status launch_chunk(const ChunkArgs &a, int64_t tiles, void *stream)
{
    static std::atomic<unsigned long long> ready[kMaxDevices];
    if (!allow_smem(weigh_chunk_kernel<CODE, D>, ready, Chunk<D>::kSmem)) return KVL_ECUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    weigh_rows_prepare_kernel<TYPE, D><<<dim3(unsigned(tiles), unsigned(a.w.t.cache.n_kv_heads)), 256, 0, st>>>(a);
    if (launch_status()) return KVL_ECUDA;
    return launch_behind(weigh_chunk_kernel<CODE, D>, a.sms, kThreads, Chunk<D>::kSmem, stream, a);
}

template <int CODE, int TYPE>
kvl_status launch_chunk_dim(const ChunkArgs &a, int64_t tiles, void *stream)
{
    return a.w.t.cache.head_dim <= 64 ? launch_chunk<CODE, TYPE, 64>(a, tiles, stream) : launch_chunk<CODE, TYPE, 128>(a, tiles, stream);
}

int64_t tiles_of(int n_seq, int64_t n_rows, int G) { return n_rows * G / kRows + n_seq + 1; }

}  // namespace

size_t weigh_chunk_bytes(const kvl_cache &c, int n_seq, int64_t n_rows, int n_heads, int sms)
{
    const size_t tile = c.head_dim <= 64 ? Chunk<64>::kTileBytes : Chunk<128>::kTileBytes;
    return counter_bytes(sms) + part_bytes(sms) + size_t(tiles_of(n_seq, n_rows, n_heads / c.n_kv_heads)) * c.n_kv_heads * tile;
}

kvl_status launch_weigh_chunk(const WeighArgs &w, void *d_workspace, int sms, void *stream)
{
    ChunkArgs a;
    a.w = w;
    a.counters = static_cast<uint32_t *>(d_workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(d_workspace) + counter_bytes(sms));
    a.tiles = static_cast<uint8_t *>(d_workspace) + counter_bytes(sms) + part_bytes(sms);
    a.sms = sms;
    const int64_t tiles = tiles_of(w.t.seqs.n_seq, w.t.seqs.n_rows, w.t.attn.n_heads / w.t.cache.n_kv_heads);
    const bool bf = w.t.attn.type == KVL_TYPE_BFLOAT;
    if (w.t.cache.code_type == KVL_CODE_FLOAT)
        return bf ? launch_chunk_dim<KVL_CODE_FLOAT, KVL_TYPE_BFLOAT>(a, tiles, stream)
                  : launch_chunk_dim<KVL_CODE_FLOAT, KVL_TYPE_HALF>(a, tiles, stream);
    return bf ? launch_chunk_dim<KVL_CODE_INT, KVL_TYPE_BFLOAT>(a, tiles, stream)
              : launch_chunk_dim<KVL_CODE_INT, KVL_TYPE_HALF>(a, tiles, stream);
}

}  // namespace kvl

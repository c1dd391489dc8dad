// kvl_append.cu -- quantise fresh K and V rows into the pages of an 8-bit cache.
//
// For each (page, head) that receives rows x:  scale' = max(old scale if the page held tokens,
// max|x| * (1/qmax), 1e-30);  code = round(clamp(x * (1/scale')));  earlier codes of the page become
// round(code * (old/scale')).  Each (plane, page, head) belongs to one CTA, so nothing is
// atomic and the result is a function of the inputs alone.
//
// Bound by instructions for prompts (2 bytes read, 1 written per element), by latency for single
// tokens (256 sequences: 13 us a call, most of it the host's).  Units: entry i of the batch may touch at most floor(n_i / B) + 2 pages, so unit
// floor(starts[i] / B) + 2 i + j is its j-th page: a warp finds i by a 32-way search of starts,
// no plan or scan is needed.  A warp holds 16 slots of one head in registers, 8 elements a lane in
// each row, so the rows are read once: their largest magnitude is reduced by shuffles (and through
// shared memory when a page spans several warps), then the registers are quantised.  A lane's 8
// elements are 4 pairs of the rotary positions, so a turn needs no other lane; a page's angles are
// worked out once for all of a CTA's heads.  Pages of more than 128 tokens are read twice instead.
#include "kvl_quant.cuh"

namespace kvl {
namespace {

constexpr int kWarps = 8;
// Slots of one head a warp holds (8, so that a page of 16 takes two warps: 94 us for 31,001 tokens, 66 with 16).
constexpr int kSlotsPerWarp = 16;

struct AppendArgs {
    kvl_cache cache;
    kvl_sequences seqs;
    kvl_rows k, v;
    const float *inv_freq;  // null: K is not turned
    int32_t n_freq, interleaved;
    float gain;
    int32_t layer;
    int32_t warps_per_head;  // warps that share a page's slots of one head: 1, 2, 4 or 8
    void *report;
};

// The batch entry that unit u belongs to: the largest i with starts[i]/B + 2i <= u.
__device__ __forceinline__ int find_entry(const kvl_sequences &s, int32_t B, int64_t u, int lane)
{
    int lo = 0, hi = s.n_seq;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const bool below = i < hi && max(s.starts[i], 0) / B + 2ll * i <= u;
        const unsigned m = __ballot_sync(0xffffffffu, below);
        const int last = m ? 31 - __clz(m) : 0;
        lo += last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Four elements as they are in memory.
template <int TYPE>
struct Raw4 {
    uint32_t w[TYPE == KVL_TYPE_FLOAT ? 4 : 2];
};

template <int TYPE>
__device__ __forceinline__ Raw4<TYPE> load_raw4(const uint8_t *p)
{
    Raw4<TYPE> r;
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = x.x; r.w[1] = x.y;
    }
    return r;
}

template <int TYPE>
__device__ __forceinline__ void floats_of(const Raw4<TYPE> &r, float *v)
{
    if constexpr (TYPE == KVL_TYPE_FLOAT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (TYPE == KVL_TYPE_BFLOAT) {
                v[2 * i] = __uint_as_float(r.w[i] << 16);
                v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

// Lanes of a row: LPR, each holding 8 elements; 32 / LPR rows a vector.  Three CTAs an SM (80 registers a
// thread, past which the forms of 16 lanes spill 230 to 340 bytes and those of 8 28 to 40; even so
// 31,001 tokens of 8 heads of 128 take 59 us, 3.2 TB/s, with two 65.6, with four, which spill more, 70.7;
// 64 sequences of 100 and d = 64: 14.8, 16.8 and 14.6); rows of 32 lanes hold twice as much and get one
// (255 registers, 16 bytes spilled).
template <int TYPE, int CODE, int LPR>
__global__ void __launch_bounds__(kWarps * 32, LPR < 32 ? 3 : 1) append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int kSize = TYPE == KVL_TYPE_FLOAT ? 4 : 2;
    constexpr int kRows = 32 / LPR;                // rows per vector of a warp
    constexpr int kVecs = kSlotsPerWarp / kRows;   // vectors per 16 slots
    constexpr float kMax = CODE == KVL_CODE_FLOAT ? 448.f : 127.f;
    extern __shared__ __align__(16) float turns[];  // cosines, then sines: [slots of a pass][n_freq] each
    __shared__ float s_amax[kWarps];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t B = a.cache.block_tokens, H = a.cache.n_kv_heads, d = a.cache.head_dim;
    const int i = find_entry(a.seqs, B, blockIdx.x, lane);
    const Entry e = load_entry(a.seqs, B, i, threadIdx.x == 0 ? a.report : nullptr);
    const int64_t j = blockIdx.x - (int64_t(e.row0) / B + 2ll * i);
    const int32_t pos0 = e.len - e.fresh;
    if (e.fresh > 0 && pos0 < 0) {
        if (threadIdx.x == 0) report(a.report, KVL_EINVAL, i);
        return;
    }
    const int32_t blk = pos0 / B + int32_t(j);
    if (e.fresh <= 0 || j < 0 || int64_t(blk) * B >= e.len) return;
    const int32_t page = e.table[blk];            // looked at after the rows' loads are on their way
    const int plane = blockIdx.y & 1;
    const int heads_per_cta = kWarps / a.warps_per_head;
    const int h = int(blockIdx.y >> 1) * heads_per_cta + warp / a.warps_per_head;
    const int part = warp % a.warps_per_head;     // which 16 slots of a pass this warp takes
    const int pass_slots = a.warps_per_head * kSlotsPerWarp;
    const int32_t page_pos = blk * B;             // cache position of slot 0
    const int s0 = max(pos0 - page_pos, 0);       // fresh slots [s0, s1)
    const int s1 = min(B, e.len - page_pos);
    const bool turn = plane == 0 && a.inv_freq != nullptr;
    const bool mine = h < H;

    // This lane's elements of a row, two runs of four: 4 pairs of the halves (e0 and e0 + n_freq), or 8 in a row.
    const int l = lane % LPR, quads = a.n_freq / 4;
    const bool halves = turn && !a.interleaved;
    const int e0 = halves && l < quads ? 4 * l : 8 * l;
    const int e1 = halves && l < quads ? a.n_freq + 4 * l : e0 + 4;
    const int pair0 = 4 * l;                      // its first pair
    const bool turns_here = turn && l < quads;
    const bool in_row = 8 * l < d;
    const kvl_rows src = plane ? a.v : a.k;
    const int slot_in = part * kSlotsPerWarp + lane / LPR;
    const uint8_t *rows = static_cast<const uint8_t *>(src.data) + int64_t(mine ? h : 0) * src.head_stride +
                          (int64_t(e.row0) - pos0 + page_pos + slot_in) * src.row_stride;

    const int passes = (s1 + pass_slots - 1) / pass_slots;
    const int first_pass = s0 / pass_slots;
    float v[kVecs][8];
    auto load_pass = [&](int pass) {
        const int base = pass * pass_slots;
        Raw4<TYPE> x0[kVecs], x1[kVecs];
#pragma unroll
        for (int n = 0; n < kVecs; ++n) {
            const int slot = base + slot_in + n * kRows;
            x0[n] = x1[n] = Raw4<TYPE>{};
            if (mine && in_row && slot >= s0 && slot < s1) {
                const uint8_t *p = rows + (base + n * kRows) * src.row_stride;
                x0[n] = load_raw4<TYPE>(p + e0 * kSize);
                x1[n] = load_raw4<TYPE>(p + e1 * kSize);
            }
        }
        if (turn) {
            const int lo = max(base, s0), hi = min(base + pass_slots, s1);
            __syncthreads();  // readers of the previous pass
            for (int t = threadIdx.x; t < (hi - lo) * a.n_freq; t += kWarps * 32) {
                const int r = t / a.n_freq, f = t - r * a.n_freq;
                const float2 cs = cos_sin_of(page_pos + lo + r, a.inv_freq[f]);
                turns[(lo - base + r) * a.n_freq + f] = cs.x * a.gain;
                turns[(pass_slots + lo - base + r) * a.n_freq + f] = cs.y * a.gain;
            }
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < kVecs; ++n) {
            floats_of<TYPE>(x0[n], v[n]);
            floats_of<TYPE>(x1[n], v[n] + 4);
            if (!turn) continue;
            const int slot = base + slot_in + n * kRows;
            if (!turns_here || slot < s0 || slot >= s1) continue;
            const float *ct = turns + (slot - base) * a.n_freq + pair0, *st = ct + pass_slots * a.n_freq;
            const float4 c4 = *reinterpret_cast<const float4 *>(ct), s4 = *reinterpret_cast<const float4 *>(st);
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
            if (a.interleaved) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = v[n][2 * x], q = v[n][2 * x + 1];
                    v[n][2 * x] = p * cc[x] - q * ss[x];
                    v[n][2 * x + 1] = q * cc[x] + p * ss[x];
                }
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = v[n][x], q = v[n][4 + x];
                    v[n][x] = p * cc[x] - q * ss[x];
                    v[n][4 + x] = q * cc[x] + p * ss[x];
                }
            }
        }
    };

    // Largest magnitude by its bits; an infinity or a NaN (rare) makes the lane look again without them.
    uint32_t most = 0;
    for (int pass = first_pass; pass < passes; ++pass) {
        load_pass(pass);
        uint32_t here = 0;
#pragma unroll
        for (int n = 0; n < kVecs; ++n)
#pragma unroll
            for (int x = 0; x < 8; ++x) here = max(here, __float_as_uint(v[n][x]) & 0x7fffffffu);
        if (here >= 0x7f800000u) {
            here = 0;
#pragma unroll
            for (int n = 0; n < kVecs; ++n)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t m = __float_as_uint(v[n][x]) & 0x7fffffffu;
                    if (m < 0x7f800000u) here = max(here, m);
                }
        }
        most = max(most, here);
    }
    float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
    if (page < 0 || page >= a.cache.pool_blocks) {
        if (threadIdx.x == 0) report(a.report, KVL_ERANGE, i);
        return;
    }
    const int64_t plane_page = (int64_t(a.layer) * 2 + plane) * a.cache.pool_blocks + page;
    uint8_t *codes = static_cast<uint8_t *>(a.cache.codes) + (plane_page * B * H + (mine ? h : 0)) * d;
    float *scale_at = a.cache.scales + plane_page * H + (mine ? h : 0);
    const float was = s0 > 0 && mine ? *scale_at : 0.f;
    if (a.warps_per_head > 1) {
        if (lane == 0) s_amax[warp] = amax;
        __syncthreads();  // also: every warp of the head has read the old scale
        for (int w = warp - part; w < warp - part + a.warps_per_head; ++w) amax = fmaxf(amax, s_amax[w]);
    }
    const float now = fmaxf(fmaxf(was, __fmul_rn(amax, 1.f / kMax)), kTinyScale);
    __syncwarp();
    if (mine && part == 0 && lane == 0) *scale_at = now;

    const float inv = __frcp_rn(now);
    for (int pass = first_pass; pass < passes; ++pass) {
        if (passes - first_pass > 1) load_pass(pass);
#pragma unroll
        for (int n = 0; n < kVecs; ++n) {
            const int slot = pass * pass_slots + slot_in + n * kRows;
            if (mine && in_row && slot >= s0 && slot < s1) {
                uint8_t *p = codes + int64_t(slot) * H * d;
                const uint32_t w0 = to_codes4<CODE>(v[n][0] * inv, v[n][1] * inv, v[n][2] * inv, v[n][3] * inv);
                const uint32_t w1 = to_codes4<CODE>(v[n][4] * inv, v[n][5] * inv, v[n][6] * inv, v[n][7] * inv);
                *reinterpret_cast<uint32_t *>(p + e0) = w0;
                *reinterpret_cast<uint32_t *>(p + e1) = w1;
            }
        }
    }
    // the page's earlier slots under the new scale
    if (s0 > 0 && now != was && mine && in_row) {
        const float ratio = __fdiv_rn(was, now);
        for (int slot = part * kRows + lane / LPR; slot < s0; slot += a.warps_per_head * kRows) {
            uint2 *p = reinterpret_cast<uint2 *>(codes + int64_t(slot) * H * d + 8 * l);
            const uint2 old = *p;
            const uint32_t u[2] = {old.x, old.y};
            uint32_t w[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t lo, hi;
                codes_of<CODE>(u[y], lo, hi);
                const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), f1 = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                w[y] = to_codes4<CODE>(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
            }
            *p = make_uint2(w[0], w[1]);
        }
    }
}

template <int TYPE, int CODE, int LPR>
kvl_status launch_append(const AppendArgs &a, unsigned units, size_t smem, void *stream)
{
    static std::atomic<unsigned long long> ready[kMaxDevices];
    if (smem > 48 * 1024 - 1024 && !allow_smem(append_kernel<TYPE, CODE, LPR>, ready, 200 * 1024)) return KVL_ECUDA;
    const int heads_per_cta = kWarps / a.warps_per_head;
    const unsigned groups = unsigned((a.cache.n_kv_heads + heads_per_cta - 1) / heads_per_cta);
    append_kernel<TYPE, CODE, LPR><<<dim3(units, 2 * groups), kWarps * 32, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return launch_status();
}

template <int TYPE, int CODE>
kvl_status launch_append_dim(const AppendArgs &a, unsigned units, size_t smem, void *stream)
{
    // lanes of a row: the power of two that holds head_dim / 8
    if (a.cache.head_dim <= 64) return launch_append<TYPE, CODE, 8>(a, units, smem, stream);
    if (a.cache.head_dim <= 128) return launch_append<TYPE, CODE, 16>(a, units, smem, stream);
    return launch_append<TYPE, CODE, 32>(a, units, smem, stream);
}

template <int TYPE>
kvl_status launch_append_code(const AppendArgs &a, unsigned units, size_t smem, void *stream)
{
    return a.cache.code_type == KVL_CODE_FLOAT ? launch_append_dim<TYPE, KVL_CODE_FLOAT>(a, units, smem, stream)
                                               : launch_append_dim<TYPE, KVL_CODE_INT>(a, units, smem, stream);
}

__global__ void report_reset_kernel(PlanHeader *h)
{
    h->status = KVL_OK;
    h->magic = kPlanMagic;
    for (int i = 0; i < 8; ++i) h->detail[i] = ~0ull;
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" kvl_status kvl_report_reset(void *d_report, void *stream)
{
    if (!d_report) return KVL_EINVAL;
    if (!aligned16(d_report)) return KVL_EALIGN;
    report_reset_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<PlanHeader *>(d_report));
    return launch_status();
}

extern "C" kvl_status kvl_cache_append(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                                       int32_t type, const kvl_rows *k, const kvl_rows *v,
                                       const kvl_rope *rope, void *d_report, void *stream)
{
    kvl_status s = check_cache(cache);
    if (!s) s = check_sequences(seqs);
    if (s) return s;
    if (layer < 0 || layer >= cache->n_layers || type < KVL_TYPE_BFLOAT || type > KVL_TYPE_FLOAT) return KVL_EINVAL;
    if (rope && (rope->reserved != 0 || rope->n_freq <= 0 || rope->n_freq % 8 || 2 * rope->n_freq > cache->head_dim ||
                 (rope->interleaved & ~1) || !rope->inv_freq))
        return KVL_EINVAL;
    if (rope && misaligned4(rope->inv_freq)) return KVL_EALIGN;
    if (bad_report(d_report)) return KVL_EALIGN;
    if (seqs->n_seq == 0 || seqs->n_rows == 0) return KVL_OK;
    if ((s = check_rows(k)) || (s = check_rows(v))) return s;
    const int32_t B = cache->block_tokens;
    AppendArgs a;
    a.cache = *cache;
    a.seqs = *seqs;
    a.k = *k;
    a.v = *v;
    a.inv_freq = rope ? rope->inv_freq : nullptr;
    a.n_freq = rope ? rope->n_freq : 0;
    a.interleaved = rope ? rope->interleaved : 0;
    a.gain = rope ? rope->gain : 1.f;
    a.layer = layer;
    a.report = d_report;
    a.warps_per_head = 1;
    while (a.warps_per_head < kWarps && a.warps_per_head * kSlotsPerWarp < B) a.warps_per_head *= 2;
    const int64_t units = seqs->n_rows / B + 2ll * seqs->n_seq;
    const size_t smem = size_t(2) * a.warps_per_head * kSlotsPerWarp * a.n_freq * sizeof(float);
    if (type == KVL_TYPE_BFLOAT) return launch_append_code<KVL_TYPE_BFLOAT>(a, unsigned(units), smem, stream);
    if (type == KVL_TYPE_HALF) return launch_append_code<KVL_TYPE_HALF>(a, unsigned(units), smem, stream);
    return launch_append_code<KVL_TYPE_FLOAT>(a, unsigned(units), smem, stream);
}

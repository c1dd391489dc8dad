// kvl_attend_shared.cu -- attention of a batch whose sequences share prefixes: each group's shared tokens once for the
// rows of all its sequences, every sequence's own tokens, and the join of both.
//
// A softmax over [0, len) is the join of those over [0, P) and [P, len): with references m1, m2, sums l1, l2 and
// weighted values O1, O2, m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), O likewise; so of any number of parts.
//   own tokens      the few-rows kernel, a row's (m, l, O) each; for groups of few rows it takes the shared tokens in
//                   the same launch, as entries of their own
//   shared tokens   of groups of more rows, the tensor-memory kernel; a (group, KV head, 256 rows) is cut over CTAs and
//                   each leaves a part.  Nothing of it waits for the kernel before, beside whose end it starts
//   join            a warp a row and head: the parts in the order of the CTAs, then the row's own tokens
#include "kvl_attend.cuh"

namespace kvl {
namespace {

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

int workspace_sms()
{
    const int n = sm_count();
    return n > 0 ? n : 152;
}

// What d_parts holds.
struct Layout {
    bool few;
    int64_t jobs, most;  // entries of the tensor-memory kernel's job table, its parts
    size_t sharing, row_ml, row_o, part_jobs, parts, bytes;
};

Layout layout_of(const kvl_cache &c, int n_seq, int n_groups, int64_t n_rows, int n_heads)
{
    Layout l = {};
    const int D = padded_dim(c.head_dim), G = n_heads / c.n_kv_heads;
    // Rows of a group (fresh tokens x query heads of a KV head) on average.  Both kernels (us, few rows / tensor memory;
    // 8 KV heads of 128, prefix of 30,000): 16 rows 34 / 54, 32 43 / 54, 48 53 / 55, 64 64 / 55, 128 109 / 58; 16 groups
    // on 2,000 32 rows 72 / 85, 48 108 / 98, 64 135 / 110; 48 of 18 on 2,600 (4 heads of 64) 67 / 102.
    l.few = c.head_dim > 128 || n_rows * G <= int64_t(kChunkRows) * n_groups;
    const size_t rows = size_t(n_rows) * n_heads * (l.few ? 2 : 1);
    l.sharing = 16;
    l.row_o = l.sharing + size_t(n_seq) * sizeof(Sharing);
    l.row_ml = l.row_o + rows * D * 4;
    l.bytes = l.row_ml + rows * 8;
    if (!l.few) {
        l.jobs = (n_rows * G / kChunkJobRows + n_groups + 1) * c.n_kv_heads;
        l.most = l.jobs + workspace_sms();
        l.part_jobs = (l.bytes + 15) & ~size_t(15);
        l.parts = (l.part_jobs + size_t(l.jobs) * 8 + 15) & ~size_t(15);
        l.bytes = l.parts + size_t(l.most) * kChunkJobRows * (D + 2) * 4 + 16;  // (to begin on 32 bytes)
    }
    return l;
}

constexpr int kThreads = 256;

// A warp (half a warp at head_dim 64) a row and head.  Its lanes look for the row's entry together, weigh a part each,
// and add up four elements of every part.
template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ AttendArgs a)
{
    constexpr int kLanes = D / 4 < 32 ? D / 4 : 32, kVecs = D / 4 / kLanes;
    const int lane = threadIdx.x % kLanes, at = lane * 4, shift = int(threadIdx.x & 31) - lane;
    const unsigned mine = (kLanes == 32 ? 0xffffffffu : (1u << kLanes) - 1) << shift;  // (rows' lanes go their own way)
    const int64_t unit = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int heads = a.attn.n_heads, n_seq = a.seqs.n_seq;
    const int64_t t = unit / heads;
    const int head = int(unit - t * heads);
    // the row's entry: the last that starts at t or before (looked for while the kernels before run)
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int step = (hi - lo + kLanes - 1) / kLanes, i = lo + lane * step;
        const unsigned below = __ballot_sync(mine, i < hi && a.seqs.starts[i] <= t) >> shift;
        const int last = below ? 31 - __clz(below) : 0;
        lo += last * step;
        hi = min(hi, lo + step);
    }
    const bool there = t < a.seqs.n_rows && t >= a.seqs.starts[lo] && t < a.seqs.starts[lo + 1];
    grid_dependency_wait();
    const Sharing s = reinterpret_cast<const Sharing *>(a.sharing)[lo];
    const bool done = a.parts_done[0] != 0 && (a.few || a.parts_done[1] != 0);
    if (!there || !done || s.tokens < 0 || (s.tokens > 0 && a.parts_done[2] != 0)) return;
    const int64_t row = t * heads + head;
    const float2 own = *reinterpret_cast<const float2 *>(a.row_ml + row * 2);
    float4 v[kVecs];
#pragma unroll
    for (int x = 0; x < kVecs; ++x) v[x] = *reinterpret_cast<const float4 *>(a.row_o + row * D + at + x * 128);
    // the shared tokens' parts
    const float *ml = nullptr, *o = nullptr;
    int parts = 0, to_sum = 1;  // from a reference to its sum
    int64_t step = 0;
    if (s.tokens > 0 && a.few) {
        const int64_t r = row + a.seqs.n_rows * heads;
        ml = a.row_ml + r * 2;
        o = a.row_o + r * D;
        parts = 1;
    } else if (s.tokens > 0) {
        const int H = a.cache.n_kv_heads, G = heads / H, h = head / G;
        const int64_t in = (t - s.row0) * G + head % G, tile = in / kChunkJobRows, r = in - tile * kChunkJobRows;
        const int2 j = reinterpret_cast<const int2 *>(a.part_jobs)[(int64_t(s.row0) * G / kChunkJobRows + s.group + tile) * H + h];
        if (j.x < 0 || j.y < 0 || j.x > a.parts_most - j.y) return;  // (no read past the parts, whatever the table holds)
        parts = j.y;
        step = int64_t(kChunkJobRows) * (D + 2);
        ml = a.group_parts + j.x * step + r;
        o = ml - r + 2 * kChunkJobRows + r * D;
        to_sum = kChunkJobRows;
    }
    float m = own.x;
    for (int b = lane; b < parts; b += kLanes) m = fmaxf(m, ml[b * step]);
#pragma unroll
    for (int x = kLanes / 2; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(mine, m, x));
    float sum = 0.f;
    float4 all[kVecs];
#pragma unroll
    for (int x = 0; x < kVecs; ++x) all[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < parts; base += kLanes) {
        const bool here = base + lane < parts;
        const float mb = here ? ml[(base + lane) * step] : -INFINITY;
        const float f = mb == -INFINITY ? 0.f : exp2_of(mb - m);
        sum += here ? ml[(base + lane) * step + to_sum] * f : 0.f;
        const int n = min(kLanes, parts - base);
        const float *p = o + base * step + at;
#pragma unroll 8
        for (int b = 0; b < n; ++b) {
            const float fb = __shfl_sync(mine, f, b, kLanes);
#pragma unroll
            for (int x = 0; x < kVecs; ++x) {
                const float4 y = *reinterpret_cast<const float4 *>(p + b * step + x * 128);
                all[x].x += y.x * fb; all[x].y += y.y * fb; all[x].z += y.z * fb; all[x].w += y.w * fb;
            }
        }
    }
#pragma unroll
    for (int x = kLanes / 2; x; x >>= 1) sum += __shfl_xor_sync(mine, sum, x);
    const float f = own.x == -INFINITY ? 0.f : exp2_of(own.x - m);
    sum += own.y * f;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int d = a.cache.head_dim;
    uint8_t *dst = static_cast<uint8_t *>(a.attn.out.data) + t * a.attn.out.row_stride + int64_t(head) * a.attn.out.head_stride;
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
        const int i = at + x * 128;
        if (i < d)
            *reinterpret_cast<uint2 *>(dst + 2 * i) = make_uint2(pack2<TYPE>((all[x].x + v[x].x * f) * inv, (all[x].y + v[x].y * f) * inv),
                                                                 pack2<TYPE>((all[x].z + v[x].z * f) * inv, (all[x].w + v[x].w * f) * inv));
    }
    if (a.attn.lse && lane == 0) a.attn.lse[row] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * (1.f / kLog2e);
}

int64_t join_ctas(const kvl_cache &c, int64_t n_rows, int n_heads)
{
    const int D = padded_dim(c.head_dim);
    return ceil_div64(n_rows * n_heads * (D / 4 < 32 ? D / 4 : 32), kThreads);
}

template <int TYPE>
kvl_status launch_join(const AttendArgs &a, void *stream)
{
    const int D = padded_dim(a.cache.head_dim);
    const int64_t ctas = join_ctas(a.cache, a.seqs.n_rows, a.attn.n_heads);
    return launch_behind(D == 64 ? join_kernel<TYPE, 64> : D == 128 ? join_kernel<TYPE, 128> : join_kernel<TYPE, 256>,
                         unsigned(ctas), kThreads, 0, stream, a);
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" size_t kvl_attend_shared_parts_bytes(const kvl_cache *cache, int32_t n_seq, int32_t n_groups, int64_t n_rows,
                                                int32_t n_heads)
{
    if (check_cache(cache) != KVL_OK || n_seq < 0 || n_seq > (1 << 20) || n_groups < 0 || n_groups > (1 << 20) || n_rows < 0 ||
        n_rows > INT32_MAX || n_heads <= 0 || n_heads > 65535 || n_heads % cache->n_kv_heads)
        return 0;
    const Layout l = layout_of(*cache, n_seq, n_groups, n_rows, n_heads);
    return l.most > INT32_MAX ? 0 : l.bytes;
}

extern "C" kvl_status kvl_attend_shared(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                                        const kvl_shared *shared, const kvl_attention *attn, void *d_workspace,
                                        size_t workspace_bytes, void *d_parts, size_t parts_bytes, void *d_report,
                                        void *stream)
{
    bool nothing = false;
    kvl_status s = check_attend(cache, layer, seqs, attn, d_workspace, workspace_bytes, d_report, &nothing);
    if (s) return s;
    if (!shared || shared->n_groups < 0 || shared->n_groups > (1 << 20) || shared->reserved != 0 ||
        (shared->n_groups > 0 && (!shared->groups || !shared->tokens)))
        return KVL_EINVAL;
    if (misaligned4(shared->groups) || misaligned4(shared->tokens) || !aligned16(d_parts)) return KVL_EALIGN;
    if (nothing) return KVL_OK;
    // What this does not serve reads its own tables: entries of more rows, whose own tokens would want the tensor-memory
    // kernel, and windows, whose rows do not all see all shared tokens (those longer than the sequences too).  From 256
    // rows an entry on nothing would be gained, as one fills a job of that kernel; below, a prefix is walked once an entry.
    const int G = attn->n_heads / cache->n_kv_heads;
    const int64_t bound = attn->max_new > 0 && attn->max_new < seqs->n_rows ? attn->max_new : seqs->n_rows;
    if (shared->n_groups == 0 || attn->window > 0 || bound * G > KVL_SHARED_ROWS)
        return kvl_attend(cache, layer, seqs, attn, d_workspace, workspace_bytes, d_report, stream);
    if (!d_parts || parts_bytes < kvl_attend_shared_parts_bytes(cache, seqs->n_seq, shared->n_groups, seqs->n_rows, attn->n_heads))
        return KVL_EINVAL;
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    if (join_ctas(*cache, seqs->n_rows, attn->n_heads) > INT32_MAX) return KVL_EINVAL;
    const Layout l = layout_of(*cache, seqs->n_seq, shared->n_groups, seqs->n_rows, attn->n_heads);
    if (l.most > INT32_MAX) return KVL_EINVAL;
    uint8_t *base = static_cast<uint8_t *>(d_parts);
    AttendArgs a = attend_args(cache, layer, seqs, attn, d_workspace, d_report);
    a.shared = *shared;
    a.parts_done = static_cast<int32_t *>(d_parts);
    a.sharing = reinterpret_cast<int32_t *>(base + l.sharing);
    a.row_o = reinterpret_cast<float *>(base + l.row_o);
    a.row_ml = reinterpret_cast<float *>(base + l.row_ml);
    a.few = l.few;
    s = launch_attend_row_parts(a, l.few ? seqs->n_rows * G : bound * G, sms, stream);
    if (!s && !l.few) {
        a.part_jobs = reinterpret_cast<int32_t *>(base + l.part_jobs);
        a.group_parts = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(base + l.parts) + 31) & ~uintptr_t(31));
        a.parts_most = int32_t(l.most);
        s = launch_attend_chunk_groups(a, sms, stream);
    }
    if (s) return s;
    return attn->type == KVL_TYPE_BFLOAT ? launch_join<KVL_TYPE_BFLOAT>(a, stream) : launch_join<KVL_TYPE_HALF>(a, stream);
}

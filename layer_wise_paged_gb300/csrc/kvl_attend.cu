// kvl_attend.cu -- attention over an 8-bit paged cache.
//
// One warp a (row, query head): one pass over the visible tokens with the running maximum and
// sum of the softmax.
#include "kvl_quant.cuh"

namespace kvl {
namespace {

constexpr int kWarps = 4;

struct AttendArgs {
    kvl_cache cache;
    kvl_sequences seqs;
    kvl_attention attn;
    int32_t layer;
    void *report;
};

template <int CODE, int TYPE>
__global__ void __launch_bounds__(kWarps * 32) attend_simple_kernel(const __grid_constant__ AttendArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int Hq = a.attn.n_heads, H = a.cache.n_kv_heads, d = a.cache.head_dim, B = a.cache.block_tokens;
    const int64_t row = unit / Hq;
    const int head = int(unit - row * Hq);
    if (row >= a.seqs.n_rows) return;
    // the entry that holds the row
    int lo = 0, hi = a.seqs.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.seqs.starts[mid] <= row) lo = mid; else hi = mid;
    }
    const Entry e = load_entry(a.seqs, B, lo, lane == 0 ? a.report : nullptr);
    if (row < e.row0 || row >= e.row0 + e.fresh) return;
    const int h = head / (Hq / H);
    const int pos = e.len - e.fresh + int(row - e.row0);
    const int j1 = a.attn.causal ? min(e.len, pos + 1) : e.len;
    const int j0 = a.attn.window > 0 ? max(0, pos - a.attn.window + 1) : 0;
    const uint16_t *q = reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(a.attn.q.data) +
                                                           row * a.attn.q.row_stride + head * a.attn.q.head_stride);
    float qv[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int x = lane + 32 * i;
        o[i] = 0.f;
        qv[i] = 0.f;
        if (x < d)
            qv[i] = TYPE == KVL_TYPE_BFLOAT ? __uint_as_float(uint32_t(q[x]) << 16) : __half2float(__ushort_as_half(q[x]));
    }
    const int64_t N = a.cache.pool_blocks, plane = int64_t(a.layer) * 2 * N;
    const uint8_t *codes = static_cast<const uint8_t *>(a.cache.codes);
    float m = -INFINITY, l = 0.f;
    for (int j = j0; j < j1; ++j) {
        const int32_t page = e.table[j / B];
        if (page < 0 || page >= N) {
            if (lane == 0) report(a.report, KVL_ERANGE, lo);
            continue;
        }
        const int64_t kat = (((plane + page) * B + j % B) * H + h) * d, vat = kat + N * B * H * d;
        const float ks = a.cache.scales[(plane + page) * H + h], vs = a.cache.scales[(plane + N + page) * H + h];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < d) s = fmaf(qv[i], of_code<CODE>(codes[kat + lane + 32 * i]), s);
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= ks * a.attn.sm_scale;
        const float mn = fmaxf(m, s);
        const float c = expf(m - mn), p = expf(s - mn);
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane + 32 * i < d) o[i] = o[i] * c + p * vs * of_code<CODE>(codes[vat + lane + 32 * i]);
        m = mn;
    }
    uint16_t *out = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(a.attn.out.data) +
                                                 row * a.attn.out.row_stride + head * a.attn.out.head_stride);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < d) out[lane + 32 * i] = uint16_t(pack2<TYPE>(j1 > j0 ? o[i] / l : 0.f, 0.f));
    if (a.attn.lse && lane == 0) a.attn.lse[row * Hq + head] = m + logf(l);
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" size_t kvl_attend_workspace_bytes(const kvl_cache *cache)
{
    return check_cache(cache) == KVL_OK ? KVL_ATTEND_ZERO_BYTES : 0;
}

extern "C" kvl_status kvl_attend(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                                 const kvl_attention *attn, void *d_workspace, size_t workspace_bytes,
                                 void *d_report, void *stream)
{
    kvl_status s = check_cache(cache);
    if (!s) s = check_sequences(seqs);
    if (s) return s;
    if (!attn || layer < 0 || layer >= cache->n_layers) return KVL_EINVAL;
    if (attn->n_heads <= 0 || attn->n_heads > 65535 || attn->n_heads % cache->n_kv_heads ||
        (attn->type != KVL_TYPE_BFLOAT && attn->type != KVL_TYPE_HALF) || !(attn->sm_scale > 0.f && attn->sm_scale < INFINITY) ||
        (attn->causal & ~1) || attn->window < 0 || (attn->window > 0 && !attn->causal) || attn->max_new < 0)
        return KVL_EINVAL;
    if (bad_report(d_report)) return KVL_EALIGN;
    if (seqs->n_seq == 0 || seqs->n_rows == 0) return KVL_OK;
    if ((s = check_rows(&attn->q)) || (s = check_rows(&attn->out))) return s;
    if (misaligned4(attn->lse) || !aligned16(d_workspace)) return KVL_EALIGN;
    if (!d_workspace || workspace_bytes < kvl_attend_workspace_bytes(cache)) return KVL_EINVAL;
    AttendArgs a = {*cache, *seqs, *attn, layer, d_report};
    const int64_t units = seqs->n_rows * attn->n_heads;
    const unsigned grid = unsigned((units + kWarps - 1) / kWarps);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->code_type == KVL_CODE_FLOAT) {
        if (attn->type == KVL_TYPE_BFLOAT) attend_simple_kernel<KVL_CODE_FLOAT, KVL_TYPE_BFLOAT><<<grid, kWarps * 32, 0, st>>>(a);
        else attend_simple_kernel<KVL_CODE_FLOAT, KVL_TYPE_HALF><<<grid, kWarps * 32, 0, st>>>(a);
    } else {
        if (attn->type == KVL_TYPE_BFLOAT) attend_simple_kernel<KVL_CODE_INT, KVL_TYPE_BFLOAT><<<grid, kWarps * 32, 0, st>>>(a);
        else attend_simple_kernel<KVL_CODE_INT, KVL_TYPE_HALF><<<grid, kWarps * 32, 0, st>>>(a);
    }
    return launch_status();
}

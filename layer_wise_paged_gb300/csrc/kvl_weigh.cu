// kvl_weigh.cu -- the entry points that weigh cached tokens: checks, choice of kernel.
#include <cmath>

#include "kvl_weigh.cuh"

using namespace kvl;

namespace {

// Entries of more rows than this (fresh tokens x query heads of a KV head; of those the call's bound allows, without one
// the average) go to the tensor-memory kernel, which takes its time for 128 of them, the few-rows kernel for each 16.
// Measured (us, few rows / tensor memory, 8 KV heads of 128): 32 sequences of 2,000 8 rows 30 / 65, 16 43 / 67, 32
// 82 / 66; one of 30,000 16 rows 23 / 31, 32 41 / 31.
constexpr int kChunkRowsOfWeigh = 16;
// (Past this many rows a KV head's steps would outlast the kernel's bounded waits.)
constexpr int64_t kMostChunkRows = int64_t(1) << 26;

bool by_chunks(const kvl_cache &c, int n_seq, int64_t n_rows, int n_heads, int max_new)
{
    const int64_t G = n_heads / c.n_kv_heads;
    const bool many = max_new > 0 ? (max_new < n_rows ? max_new : n_rows) * G > kChunkRowsOfWeigh : n_rows * G > int64_t(kChunkRowsOfWeigh) * n_seq;
    return c.head_dim <= 128 && many && n_rows * G <= kMostChunkRows;
}

int workspace_sms()
{
    const int n = sm_count();
    return n > 0 ? n : 152;
}

}  // namespace

extern "C" size_t kvl_weigh_workspace_bytes(const kvl_cache *cache, int32_t n_seq, int64_t n_rows, int32_t n_heads,
                                            int32_t max_new)
{
    if (check_cache(cache) != KVL_OK || n_seq < 0 || n_rows < 0 || n_rows > INT32_MAX || n_heads <= 0 || n_heads > 65535 ||
        max_new < 0)
        return 0;
    return by_chunks(*cache, n_seq, n_rows, n_heads, max_new) ? weigh_chunk_bytes(*cache, n_seq, n_rows, n_heads, workspace_sms()) : 16;
}

extern "C" kvl_status kvl_weigh(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                                const kvl_weighing *w, void *d_workspace, size_t workspace_bytes, void *d_report,
                                void *stream)
{
    kvl_status s = check_cache(cache);
    if (!s) s = check_sequences(seqs);
    if (s) return s;
    if (!w || layer < 0 || layer >= cache->n_layers) return KVL_EINVAL;
    if (w->n_heads <= 0 || w->n_heads > 65535 || w->n_heads % cache->n_kv_heads ||
        (w->type != KVL_TYPE_BFLOAT && w->type != KVL_TYPE_HALF) || !(w->sm_scale > 0.f && w->sm_scale < INFINITY) ||
        (w->causal & ~1) || w->window < 0 || (w->window > 0 && !w->causal) || w->max_new < 0 || (w->begin & ~1) || w->reserved != 0)
        return KVL_EINVAL;
    if (seqs->n_rows * (w->n_heads / cache->n_kv_heads) > INT32_MAX - 256) return KVL_EINVAL;
    if (bad_report(d_report)) return KVL_EALIGN;
    if (seqs->n_seq == 0 || seqs->n_rows == 0) return KVL_OK;
    if ((s = check_rows(&w->q))) return s;
    if (!w->lse || !w->mass_in || !w->mass_out || w->tokens <= 0 || w->in_stride < w->tokens || w->out_stride < w->tokens) return KVL_EINVAL;
    if (misaligned4(w->lse) || misaligned4(w->mass_in) || misaligned4(w->mass_out) || !aligned16(d_workspace)) return KVL_EALIGN;
    if (!d_workspace || workspace_bytes < kvl_weigh_workspace_bytes(cache, seqs->n_seq, seqs->n_rows, w->n_heads, w->max_new))
        return KVL_EINVAL;
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    WeighArgs a = {};
    a.t.cache = *cache;
    a.t.seqs = *seqs;
    a.t.layer = layer;
    a.t.report = d_report;
    a.t.attn.q = w->q;
    a.t.attn.n_heads = w->n_heads;
    a.t.attn.type = w->type;
    a.t.attn.sm_scale = w->sm_scale;
    a.t.attn.causal = w->causal;
    a.t.attn.window = w->window;
    a.lse = w->lse;
    a.mass_in = w->mass_in;
    a.mass_out = w->mass_out;
    a.in_stride = w->in_stride;
    a.out_stride = w->out_stride;
    a.tokens = w->tokens;
    a.begin = w->begin;
    if (by_chunks(*cache, seqs->n_seq, seqs->n_rows, w->n_heads, w->max_new)) return launch_weigh_chunk(a, d_workspace, sms, stream);
    const int64_t bound = w->max_new > 0 && w->max_new < seqs->n_rows ? w->max_new : seqs->n_rows;
    return launch_weigh_rows(a, bound * (w->n_heads / cache->n_kv_heads), sms, stream);
}

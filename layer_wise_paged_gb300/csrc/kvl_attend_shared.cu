// kvl_attend_shared.cu -- attention of a batch whose sequences share prefixes: each group's shared tokens once for
// the rows of all its sequences, then every sequence's own tokens, joined with what the shared ones gave.
//
// A softmax over [0, len) is the join of those over [0, P) and [P, len): with references m1, m2, sums l1, l2 and
// weighted values O1, O2, m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), O likewise.
#include "kvl_attend_rows.cuh"

using namespace kvl;

namespace {

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

}  // namespace

extern "C" size_t kvl_attend_shared_parts_bytes(const kvl_cache *cache, int64_t n_rows, int32_t n_heads)
{
    if (check_cache(cache) != KVL_OK || n_rows < 0 || n_rows > INT32_MAX || n_heads <= 0 || n_heads > 65535) return 0;
    return size_t(n_rows) * n_heads * (padded_dim(cache->head_dim) + 2) * sizeof(float) + 16;
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
    if (!d_parts || parts_bytes < kvl_attend_shared_parts_bytes(cache, seqs->n_rows, attn->n_heads)) return KVL_EINVAL;
    // With a window most rows see little of a long prefix, and entries of many rows are bound by the products, which
    // sharing does not spare: both read their own tables.
    const int G = attn->n_heads / cache->n_kv_heads;
    const int64_t bound = attn->max_new > 0 && attn->max_new < seqs->n_rows ? attn->max_new : seqs->n_rows;
    if (shared->n_groups == 0 || attn->window > 0 || bound * G > kChunkRows)
        return kvl_attend(cache, layer, seqs, attn, d_workspace, workspace_bytes, d_report, stream);
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    AttendArgs a = attend_args(cache, layer, seqs, attn, d_workspace, d_report);
    a.shared = *shared;
    a.row_o = static_cast<float *>(d_parts);
    a.row_ml = a.row_o + size_t(seqs->n_rows) * attn->n_heads * padded_dim(cache->head_dim);
    s = launch_rows_part<Part::shared>(a, seqs->n_rows * G, sms, stream);
    return s ? s : launch_rows_part<Part::own>(a, bound * G, sms, stream);
}

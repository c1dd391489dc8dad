// kvl_attend_shared.cu -- attention of a batch whose sequences share prefixes: each group's shared tokens once for
// the rows of all its sequences, then every sequence's own tokens, joined with what the shared ones gave.
//
// A softmax over [0, len) is the join of those over [0, P) and [P, len): with references m1, m2, sums l1, l2 and
// weighted values O1, O2, m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), O likewise.
#include "kvl_attend_rows.cuh"

using namespace kvl;

namespace {

int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// Groups of so many rows on average (fresh tokens x query heads of a KV head) go to the few-rows kernel.
constexpr int64_t kFewRows = 16;

int workspace_sms()
{
    const int n = sm_count();
    return n > 0 ? n : 152;
}

// What d_parts holds: a flag, every entry's sharing, then rows' results, or the tensor-memory kernel's job table and parts.
struct Layout {
    int rows;              // of a tile of the tensor-memory kernel; 0: few rows
    int64_t jobs, most;    // entries of the job table, parts
    size_t sharing, first, second;  // offsets of the sharing, of row_o and row_ml, or of the table and the parts
    size_t bytes;
};

Layout layout_of(const kvl_cache &c, int n_seq, int n_groups, int64_t n_rows, int n_heads)
{
    Layout l = {};
    const int D = padded_dim(c.head_dim), G = n_heads / c.n_kv_heads, sms = workspace_sms();
    l.sharing = 16;
    l.first = l.sharing + size_t(n_seq) * sizeof(Sharing);
    if (c.head_dim > 128 || n_rows * G <= kFewRows * n_groups || sms > kMostParts) {
        l.second = l.first + size_t(n_rows) * n_heads * D * 4;
        l.bytes = l.second + size_t(n_rows) * n_heads * 8;
        return l;
    }
    l.rows = n_rows * G <= int64_t(kPrefixTileRows) * n_groups ? kPrefixTileRows : kChunkTileRows;
    l.jobs = prefix_tiles(n_rows, G, n_groups, l.rows) * c.n_kv_heads;
    l.most = l.jobs + sms;
    l.second = (l.first + size_t(l.jobs) * 8 + 15) & ~size_t(15);
    l.bytes = l.second + size_t(l.most) * l.rows * (D + 2) * 4;
    return l;
}

}  // namespace

extern "C" size_t kvl_attend_shared_parts_bytes(const kvl_cache *cache, int32_t n_seq, int32_t n_groups, int64_t n_rows,
                                                int32_t n_heads)
{
    if (check_cache(cache) != KVL_OK || n_seq < 0 || n_seq > (1 << 20) || n_groups < 0 || n_groups > (1 << 20) || n_rows < 0 || n_rows > INT32_MAX || n_heads <= 0 ||
        n_heads > 65535 || n_heads % cache->n_kv_heads)
        return 0;
    return layout_of(*cache, n_seq, n_groups, n_rows, n_heads).bytes;
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
    if (!d_parts || parts_bytes < kvl_attend_shared_parts_bytes(cache, seqs->n_seq, shared->n_groups, seqs->n_rows, attn->n_heads)) return KVL_EINVAL;
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
    const Layout l = layout_of(*cache, seqs->n_seq, shared->n_groups, seqs->n_rows, attn->n_heads);
    uint8_t *base = static_cast<uint8_t *>(d_parts);
    a.shared_done = static_cast<int32_t *>(d_parts);
    a.sharing = reinterpret_cast<int32_t *>(base + l.sharing);
    if (l.rows == 0) {
        a.row_o = reinterpret_cast<float *>(base + l.first);
        a.row_ml = reinterpret_cast<float *>(base + l.second);
        s = launch_rows_part<Part::shared>(a, seqs->n_rows * G, sms, stream);
    } else {
        a.prefix_rows = l.rows;
        a.prefix_most = int32_t(l.most);
        a.prefix_jobs = reinterpret_cast<int32_t *>(base + l.first);
        a.prefix_parts = reinterpret_cast<float *>(base + l.second);
        s = l.rows == kPrefixTileRows ? launch_attend_prefix(a, sms, stream) : launch_attend_chunk_shared(a, sms, stream);
    }
    return s ? s : launch_rows_part<Part::own>(a, bound * G, sms, stream);
}

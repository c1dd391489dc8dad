// kvl_attend.cu -- the entry points of attention over an 8-bit paged cache: checks, workspace,
// choice of kernel.
#include <cmath>

#include "kvl_attend.cuh"

namespace kvl {
namespace {

// Why kChunkRows is 40: the tensor-memory kernel's time hardly depends on the rows up to 256, while attend_rows'
// grows with each 16.  Measured
// (us, rows / chunk; 8 KV heads, e4m3; int8 the same within 3 %):
//   32 sequences of 2,048 tokens   d = 128: 32 rows 85 / 92, 40 115 / 92, 48 116 / 93
//                                  d = 64: 16 rows 33 / 70, 32 52 / 70, 40 72 / 70, 64 90 / 70
//   one of 32,768                  d = 128: 32 rows 42 / 51, 48 54 / 51, 64 66 / 53
//                                  d = 64: 32 rows 31 / 38, 40 38 / 39, 48 37 / 39, 64 45 / 39
//   4 of 500                       40 rows, d = 128: 18 / 29, d = 64: 14 / 25
//   16 of 1,000                    36 rows, d = 128: 42 / 43, d = 64 (4 heads): 23 / 29
// At 33 to 40 rows large batches would gain up to a fifth by the chunk kernel, small ones lose a half.

// SMs the workspace is sized for (a host without a device sizes it for a GB300).
int workspace_sms()
{
    const int n = sm_count();
    return n > 0 ? n : 152;
}

}  // namespace
}  // namespace kvl

using namespace kvl;

extern "C" size_t kvl_attend_workspace_bytes(const kvl_cache *cache)
{
    if (check_cache(cache) != KVL_OK) return 0;
    const size_t rows = attend_rows_part_bytes(cache->head_dim), chunk = attend_chunk_part_bytes(cache->head_dim);
    return KVL_ATTEND_ZERO_BYTES + size_t(workspace_sms()) * (rows > chunk ? rows : chunk);
}

extern "C" uint64_t kvl_capture_id(void *stream)
{
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &id) != cudaSuccess) {
        cudaGetLastError();  // (the legacy stream beside a capture of another: not in one itself)
        return 0;
    }
    return status == cudaStreamCaptureStatusNone ? 0 : id;
}

namespace kvl {

kvl_status check_attend(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs, const kvl_attention *attn,
                        const void *d_workspace, size_t workspace_bytes, const void *d_report, bool *nothing)
{
    kvl_status s = check_cache(cache);
    if (!s) s = check_sequences(seqs);
    if (s) return s;
    if (!attn || layer < 0 || layer >= cache->n_layers) return KVL_EINVAL;
    if (attn->n_heads <= 0 || attn->n_heads > 65535 || attn->n_heads % cache->n_kv_heads ||
        (attn->type != KVL_TYPE_BFLOAT && attn->type != KVL_TYPE_HALF) || !(attn->sm_scale > 0.f && attn->sm_scale < INFINITY) ||
        (attn->causal & ~1) || attn->window < 0 || (attn->window > 0 && !attn->causal) || attn->max_new < 0)
        return KVL_EINVAL;
    if (seqs->n_rows * (attn->n_heads / cache->n_kv_heads) > INT32_MAX - 256) return KVL_EINVAL;
    if (bad_report(d_report)) return KVL_EALIGN;
    *nothing = seqs->n_seq == 0 || seqs->n_rows == 0;
    if (*nothing) return KVL_OK;
    if ((s = check_rows(&attn->q)) || (s = check_rows(&attn->out))) return s;
    if (misaligned4(attn->lse) || !aligned16(d_workspace)) return KVL_EALIGN;
    if (!d_workspace || workspace_bytes < kvl_attend_workspace_bytes(cache)) return KVL_EINVAL;
    return KVL_OK;
}

AttendArgs attend_args(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs, const kvl_attention *attn,
                       void *d_workspace, void *d_report)
{
    AttendArgs a = {};
    a.cache = *cache;
    a.seqs = *seqs;
    a.attn = *attn;
    a.layer = layer;
    a.max_rows = INT32_MAX;
    a.counters = static_cast<uint32_t *>(d_workspace);
    a.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(d_workspace) + KVL_ATTEND_ZERO_BYTES);
    a.report = d_report;
    return a;
}

}  // namespace kvl

extern "C" kvl_status kvl_attend(const kvl_cache *cache, int32_t layer, const kvl_sequences *seqs,
                                 const kvl_attention *attn, void *d_workspace, size_t workspace_bytes,
                                 void *d_report, void *stream)
{
    bool nothing = false;
    kvl_status s = check_attend(cache, layer, seqs, attn, d_workspace, workspace_bytes, d_report, &nothing);
    if (s || nothing) return s;
    const int sms = sm_count();
    if (sms <= 0) return KVL_ECUDA;
    AttendArgs a = attend_args(cache, layer, seqs, attn, d_workspace, d_report);
    // Of a batch, each entry goes to the kernel that suits its rows; where the bound on them (or the only
    // entry's rows) says that one kernel takes all, the other is not launched.
    const int64_t bound = attn->max_new > 0 && attn->max_new < seqs->n_rows ? attn->max_new : seqs->n_rows;
    const int64_t most = bound * (attn->n_heads / cache->n_kv_heads);
    if (cache->head_dim > 128 || most <= kChunkRows) return launch_attend_rows(a, most, sms, stream);
    if (seqs->n_seq == 1) {
        a.max_rows = 0;
        return launch_attend_chunk(a, sms, stream);
    }
    a.max_rows = kChunkRows;
    s = launch_attend_chunk(a, sms, stream);
    return s ? s : launch_attend_rows(a, kChunkRows, sms, stream);
}

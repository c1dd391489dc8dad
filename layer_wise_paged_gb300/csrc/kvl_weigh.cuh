// kvl_weigh.cuh -- what the kernels that weigh cached tokens share.
//
// mass'[j] = mass[j] + sum over rows and query heads of 2^(x - lse log2(e)), x = sm_scale log2(e) q.K_j, over the
// rows that see token j: the probability that attention gave it, from attention's own lse, so one pass over K is
// enough and nothing is kept between tokens.  Each token's sum is made by one CTA, or by several in a fixed
// order, in 32 bits: no atomic adds, the same bits every time.
#pragma once

#include "kvl_attend.cuh"

namespace kvl {

struct WeighArgs {
    AttendArgs t;  // cache, sequences, layer, report; of attn: q, n_heads, type, sm_scale, causal, window
    const float *lse, *mass_in;
    float *mass_out;
    int64_t in_stride, out_stride;  // floats from slot to slot
    int64_t tokens;                 // that a slot has room for
    int32_t begin;                  // fresh tokens' masses start from zero
    int32_t heads_held;             // KV heads whose Q is in shared memory at a time
};

// most: a bound on the rows (fresh tokens x query heads of a KV head) of an entry, which chooses the row tile.
kvl_status launch_weigh_rows(const WeighArgs &a, int64_t most, int sms, void *stream);
size_t weigh_chunk_bytes(const kvl_cache &c, int n_seq, int64_t n_rows, int n_heads, int sms);
kvl_status launch_weigh_chunk(const WeighArgs &a, void *d_workspace, int sms, void *stream);

}  // namespace kvl

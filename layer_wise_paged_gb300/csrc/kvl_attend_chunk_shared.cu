// kvl_attend_chunk_shared.cu -- attention of groups of many rows over the tokens they share (kvl_attend_chunk.cuh has
// the kernel).
#include "kvl_attend_chunk.cuh"

namespace kvl {

static_assert(kJobRows == kChunkJobRows, "the parts' layout");

kvl_status launch_attend_chunk_groups(const AttendArgs &a, int sms, void *stream)
{
    AttendArgs b = a;
    b.attn.causal = 0;  // every row sees all shared tokens
    b.max_rows = 0;     // of whatever number
    return launch_chunk_of<true>(b, sms, stream);
}

}  // namespace kvl

// kvl_attend_chunk.cu -- attention of many rows over whole sequences (kvl_attend_chunk.cuh has the kernel).
#include "kvl_attend_chunk.cuh"

namespace kvl {

size_t attend_chunk_part_bytes(int head_dim)
{
    return head_dim > 128 ? 0 : size_t(2) * kJobRows * ((head_dim <= 64 ? 64 : 128) + 2) * sizeof(float);
}

kvl_status launch_attend_chunk(const AttendArgs &a, int sms, void *stream) { return launch_chunk_of<false>(a, sms, stream); }

}  // namespace kvl

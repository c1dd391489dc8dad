// kvl_attend_rows.cu -- attention of few rows over whole sequences (kvl_attend_rows.cuh has the kernel).
#include "kvl_attend_rows.cuh"

namespace kvl {

size_t attend_rows_part_bytes(int head_dim)
{
    const int D = head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256, rows = head_dim <= 128 ? 16 : 8;
    return size_t(2) * kCtasPerSm * (rows * (D + 2)) * sizeof(float);
}

kvl_status launch_attend_rows(const AttendArgs &a, int64_t most, int sms, void *stream)
{
    return launch_rows_part<false>(a, most, sms, stream);
}

}  // namespace kvl

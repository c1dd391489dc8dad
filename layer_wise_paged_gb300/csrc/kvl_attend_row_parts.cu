// kvl_attend_row_parts.cu -- the parts of attention over a shared prefix that few rows make (kvl_attend_rows.cuh has the
// kernel).
#include "kvl_attend_rows.cuh"

namespace kvl {

kvl_status launch_attend_row_parts(const AttendArgs &a, int64_t most, int sms, void *stream)
{
    return launch_rows_part<true>(a, most, sms, stream);
}

}  // namespace kvl

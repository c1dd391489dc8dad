// kvl_attend_prefix.cuh -- where attention over shared tokens on the tensor cores leaves its parts.
//
// Rows of a group are taken in tiles of `rows`; tile c of group g has the number row0 * G / rows + g + c (row0 the
// group's first row), so no two meet.  jobs[number][KV head] is (first part, how many follow each other); a part is
// [rows] references, [rows] sums, then values.  Parts are numbered job + share, so there are never more than
// jobs + shares.  Two kernels make them: that of kvl_attend_prefix.cu for tiles of 64 rows, values [rows][64 or 128],
// and attend_chunk's for tiles of 256, values [16 or 32][256 rows][4].
#pragma once

#include "kvl_attend.cuh"

namespace kvl {

inline int64_t prefix_tiles(int64_t n_rows, int G, int n_groups, int rows) { return n_rows * G / rows + n_groups + 1; }

constexpr int kPrefixTileRows = 64, kChunkTileRows = 256;
kvl_status launch_attend_prefix(const AttendArgs &a, int sms, void *stream);
kvl_status launch_attend_chunk_shared(const AttendArgs &a, int sms, void *stream);

}  // namespace kvl

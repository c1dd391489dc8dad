// kvl_attend_prefix.cuh -- where attention over shared tokens on the tensor cores leaves its parts.
//
// Rows of a group are taken in tiles of `rows`; tile c of group g has the number row0 * G / rows + g + c (row0 the
// group's first row), so no two meet.  jobs[number][KV head] is (first part, how many follow each other); a part is
// [rows] references, [rows] sums, [rows][64 or 128] values.  Parts are numbered job + share, so there are never more
// than jobs + shares.
#pragma once

#include "kvl_attend.cuh"

namespace kvl {

inline int64_t prefix_tiles(int64_t n_rows, int G, int n_groups, int rows) { return n_rows * G / rows + n_groups + 1; }

// rows: 64 or 128
kvl_status launch_attend_prefix(const AttendArgs &a, int rows, int sms, void *stream);

}  // namespace kvl

// Index arithmetic of the grouped products that decides which rows, tiles and
// workgroups there are: plain integers, the same on the host, on the device
// and in a CPU test that includes this header alone.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define GROUPED_HD __host__ __device__ inline __attribute__((always_inline))
#else
#define GROUPED_HD inline
#endif

namespace gemm {
namespace grouped {

// The rows fall into G + 2 segments: the rows of no group in front, the
// groups, and the rows of no group behind.  Segment i ends at
//   end(i) = max(end(i - 1), offsets[i] clamped to 0 .. T), end(G + 1) = T,
// and starts where the one before it ends, so that the segments cover
// 0 .. T once whatever the offsets hold.
GROUPED_HD int clamp_offset(int offset, int T) { return offset < 0 ? 0 : offset > T ? T : offset; }

// Whether a segment's rows are computed: those of no group only to fill them.
GROUPED_HD bool segment_runs(int i, int G, int fill) { return i <= G + 1 && (fill || (i > 0 && i <= G)); }

// Row tiles of a segment of `rows` rows.
GROUPED_HD int segment_tiles(int rows, int bm) { return (int)(((int64_t)rows + bm - 1) / bm); }

// The most row tiles that any offsets can give: sum of ceil(rows_i / bm) over
// S segments is at most (T + S (bm - 1)) / bm, and no more than T tiles have a
// row.
GROUPED_HD int64_t most_tiles(int64_t T, int64_t G, int fill, int bm) {
  const int64_t S = G + (fill ? 2 : 0), n = (T + S * (bm - 1)) / bm;
  return S == 0 ? 0 : n < T ? n : T;
}

}  // namespace grouped
}  // namespace gemm

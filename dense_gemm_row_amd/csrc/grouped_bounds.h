// Index arithmetic of the grouped and 4-bit products that decides which rows,
// tiles and workgroups there are, and where operands of any alignment are read: plain integers, the same on the host, on the device
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

// Reads in whole pieces of `per` values wherever a row ends: by how many values
// the piece that has `left` values ahead of the row's end begins early, so that
// it ends there (the row has a whole piece; what it does not need is shifted out).
template <class I>
GROUPED_HD int piece_early(I left, int per) { return left >= per ? 0 : per - (int)left; }

// The same by position: where `width` values from n on are read in a row of
// `count` >= width.
GROUPED_HD int piece_start(int n, int count, int width) { return n < count - width ? n : count - width; }

// The byte of a row of codes where the 16 bytes with k are (k a multiple of 32;
// `padded` is the row's k, whole 32): past the row's end, the row's first ones.
GROUPED_HD int code_byte(int k, int padded) { return k < padded ? k / 2 : 0; }

// The first k of the i-th span that wave row `part` of PARTS takes, `spans`
// of them from the turn-th on; from `spans` on, a whole span past the end (`past`),
// so that a lane's whole 32 k of it are there or not.
template <int SPAN>
GROUPED_HD int past_spans(int K) { return (K + SPAN - 1) / SPAN * SPAN; }
template <int PARTS, int SPAN>
GROUPED_HD int span_start(int i, int spans, int turn, int part, int past) {
  const int j = i + turn < spans ? i + turn : i + turn - spans;
  return i < spans ? (part + j * PARTS) * SPAN : past;
}

}  // namespace grouped
}  // namespace gemm

// Internal declarations of the grouped products (include/gemm_grouped.h):
// kernel arguments, launch functions, and the search for a row tile's group.
#pragma once

#include "gemm_grouped.h"
#include "gemm_internal.h"
#include "grouped_bounds.h"

namespace gemm {
namespace grouped {

constexpr int64_t kMostGroups = 65535;

struct MatmulArgs {
  const int32_t* offsets;
  const void *X, *W;
  void* Y;
  int64_t ldx, ldw, stride_w, ldy;
  int G, T, N, K;
  int fill;
  int trans_w;
};

struct WgradArgs {
  const int32_t* offsets;
  const void *X, *dY;
  void* dW;
  int64_t ldx, ldy, ldw, stride_w;
  int G, T, K, N;
  float alpha, beta;
};

// Any operands.
hipError_t launch_general(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s);
hipError_t launch_general(int dtype, int c_dtype, const WgradArgs& a, hipStream_t s);

// The product on whichever kernel and tile is best for it (grouped_api.hip).
hipError_t launch_matmul(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s);

// 16-bit operands (DT) of whole 16-byte pieces, result of type CT, on tiles of
// SIDE x SIDE (256, 128): grouped_pipe.hip.
template <int DT, int CT, int SIDE>
hipError_t launch_pipe(const MatmulArgs& a, hipStream_t s);
template <int DT, int CT, int SIDE>
hipError_t launch_pipe(const WgradArgs& a, hipStream_t s);

// Tiles of `side` along n.
inline int64_t tiles_along(int64_t n, int side) { return (n + side - 1) / side; }
// Tiles of `side` x `side` that are likely: a group ends in half a row tile on
// average, and has one where it has a row.
inline double likely_tiles(const MatmulArgs& a, int side) {
  const double some = a.T < a.G ? a.T : a.G, m = (double)a.T / side + 0.5 * some;
  return (m > some ? m : some) * tiles_along(a.N, side);
}
inline double likely_tiles(const WgradArgs& a, int side) {
  return (double)a.G * tiles_along(a.K, side) * tiles_along(a.N, side);
}
// Whether the tiles of 128 x 128 do not have to share a CU (the product's with
// some to spare: a second round costs more): then four LDS stages, three
// slices ahead, hide what a second workgroup would.  (1000 rows, 8 groups, 2048 x
// 2048: 17.5 us with four stages, 23.8 with two; 1024 rows, 32 groups, 1024 x 1024,
// 256 tiles: 20.2 and 16.2.  Gradient of 16000 rows, 16 groups, 512 x 512: 31.9 and
// 44.0; of 75 rows a group, 1024 x 1024: 7.9 and 7.4.)
constexpr int kCus = 256;
inline bool alone(const MatmulArgs& a) { return likely_tiles(a, 128) <= 240; }
inline bool alone(const WgradArgs& a) { return likely_tiles(a, 128) <= kCus && a.T >= 384ll * a.G; }

// The product on tiles of 16 rows x 64 columns, the same operands.
hipError_t launch_few(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s);

#if defined(__HIP__)
// ---------------------------------------------------------------------------
// Prefix sums and maxima over a wave's 64 lanes, six data-parallel moves each
// (row shifts by 1, 2, 4 and 8, then the last lane of row 0 to row 1 and of
// row 2 to row 3, and of row 1 to rows 2 and 3): about 100 cycles, where the
// same through LDS permutes takes some 1500.  Values are not negative, so a
// lane that a move does not reach gets 0, neutral for both.
// ---------------------------------------------------------------------------
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int scan_add(int x) {
  x += moved<0x111, 0xf>(x);
  x += moved<0x112, 0xf>(x);
  x += moved<0x114, 0xf>(x);
  x += moved<0x118, 0xf>(x);
  x += moved<0x142, 0xa>(x);
  x += moved<0x143, 0xc>(x);
  return x;
}
__device__ __forceinline__ int larger(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ int scan_max(int x) {
  x = larger(x, moved<0x111, 0xf>(x));
  x = larger(x, moved<0x112, 0xf>(x));
  x = larger(x, moved<0x114, 0xf>(x));
  x = larger(x, moved<0x118, 0xf>(x));
  x = larger(x, moved<0x142, 0xa>(x));
  x = larger(x, moved<0x143, 0xc>(x));
  return x;
}

// What the lanes know of 64 consecutive segments: where lane l's, number
// first + l, starts and ends, and the row tiles up to and with it.
struct Segments {
  int start, end, tiles;
};
// `end` and `tiles` of the segment before the first one come in and those of
// the last one go out through `end0` and `tiles0`.
__device__ __forceinline__ Segments segments(const int32_t* offsets, int G, int T, int fill, int bm, int first,
                                             int& end0, int& tiles0) {
  const int i = first + (int)(threadIdx.x & 63);
  Segments s;
  s.end = larger(scan_max(i <= G ? clamp_offset(offsets[i], T) : T), end0);
  s.start = __builtin_amdgcn_update_dpp(end0, s.end, 0x138, 0xf, 0xf, false);  // (one lane up)
  s.tiles = tiles0 + scan_add(segment_runs(i, G, fill) ? segment_tiles(s.end - s.start, bm) : 0);
  end0 = __builtin_amdgcn_readlane(s.end, 63);
  tiles0 = __builtin_amdgcn_readlane(s.tiles, 63);
  return s;
}

// A row tile: rows row0 .. row0 + rows - 1 (rows <= bm) of group g, or
// (g < 0) of no group.
struct RowTile {
  int g, row0, rows;
};

// The row tile `rt` in the order of the rows among segments `s`, whose first
// one is `first` with `before` row tiles ahead; some lane's count passes rt.
__device__ __forceinline__ RowTile tile_among(const Segments& s, int G, int bm, int first, int before, int rt) {
  // The first lane whose running count passes rt; its own first tile is the
  // count of the lane before it.
  const int lane = (int)__builtin_ctzll(__ballot(s.tiles > rt));
  const int below = lane == 0 ? before : __builtin_amdgcn_readlane(s.tiles, lane == 0 ? 0 : lane - 1);
  const int start = __builtin_amdgcn_readlane(s.start, lane), end = __builtin_amdgcn_readlane(s.end, lane);
  const int row0 = start + (rt - below) * bm, i = first + lane;
  return {i > 0 && i <= G ? i - 1 : -1, row0, end - row0 < bm ? end - row0 : bm};
}

// All row tiles that offsets give (without offsets: one group of all rows): how
// many, and each by its number.  Every lane of the wave takes part.  Up to 62
// groups the offsets are read once.
struct RowTiles {
  const int32_t* offsets;
  int G, T, fill, bm, count;
  Segments first;
  __device__ __forceinline__ RowTiles(const int32_t* offsets_, int G_, int T_, int fill_, int bm_)
      : offsets(offsets_), G(G_), T(T_), fill(fill_), bm(bm_) {
    int end = 0;
    count = offsets ? 0 : segment_tiles(T, bm);
    if (!offsets) return;
    first = segments(offsets, G, T, fill, bm, 0, end, count);
    for (int i = 64; i < G + 2; i += 64) segments(offsets, G, T, fill, bm, i, end, count);
  }
  // Tile rt, or (from count on) none, of 0 rows.
  __device__ __forceinline__ RowTile find(int rt) const {
    if (rt >= count) return {-1, 0, 0};
    if (!offsets) return {0, rt * bm, T - rt * bm < bm ? T - rt * bm : bm};
    int end = __builtin_amdgcn_readlane(first.end, 63), tiles = __builtin_amdgcn_readlane(first.tiles, 63);
    if (rt < tiles) return tile_among(first, G, bm, 0, 0, rt);
    for (int i = 64;; i += 64) {
      const int before = tiles;
      const Segments s = segments(offsets, G, T, fill, bm, i, end, tiles);
      if (rt < tiles) return tile_among(s, G, bm, i, before, rt);
    }
  }
};

// Group g's rows [start, end).
__device__ __forceinline__ void group_rows(const int32_t* offsets, int T, int g, int& start, int& end) {
  int top = 0;
  for (int first = 0; first <= g; first += 64) {
    const int i = first + (int)(threadIdx.x & 63);
    top = larger(top, __builtin_amdgcn_readlane(scan_max(i <= g ? clamp_offset(offsets[i], T) : 0), 63));
  }
  start = top;
  end = larger(top, clamp_offset(__builtin_amdgcn_readfirstlane(offsets[g + 1]), T));
}

// The same for the group of a rank by rows, the longest one 0, up to 16 groups
// (beyond: group `rank` itself): what takes longest starts first.  (8 groups of 512
// rows on average, 2048 x 2048: 62 us in order, 51 so; 64 of 256, 1024 x 1024: 80 in
// order, 96 so: finding a rank is some 20 instructions a group.)
__device__ __forceinline__ void ranked_group(const int32_t* offsets, int T, int G, int rank, int& g, int& start, int& end) {
  g = rank;
  if (G > 16) return group_rows(offsets, T, g, start, end);
  const int lane = (int)(threadIdx.x & 63), front = clamp_offset(__builtin_amdgcn_readfirstlane(offsets[0]), T);
  const int to = larger(scan_max(lane < G ? clamp_offset(offsets[lane + 1], T) : 0), front);
  const int from = __builtin_amdgcn_update_dpp(front, to, 0x138, 0xf, 0xf, false);  // (one lane up)
  const int rows = lane < G ? to - from : -1;
  int ahead = 0;
  for (int j = 0; j < G; ++j) {
    const int other = __builtin_amdgcn_readlane(rows, j);
    ahead += other > rows || (other == rows && j < lane);
  }
  g = (int)__builtin_ctzll(__ballot(lane < G && ahead == rank));
  start = __builtin_amdgcn_readlane(from, g);
  end = __builtin_amdgcn_readlane(to, g);
}
#endif

}  // namespace grouped
}  // namespace gemm

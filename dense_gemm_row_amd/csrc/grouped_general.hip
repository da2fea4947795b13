// The grouped products for any operands: every type, alignment, stride and
// size.  A workgroup of four waves computes a 64 x 64 tile, 32 k per slice;
// each wave has 2 x 2 blocks of the 16 x 16 matrix instruction (FP32: k 4,
// binary16 and bfloat16: k 32), FP32 accumulation.
//  * Both operands stand in LDS by output row (column), k contiguous, rows 16
//    bytes longer than their values: 16 rows read 16 bytes each from distinct
//    banks.  A thread stages 8 consecutive k of one row, so that its LDS write
//    is one or two 16-byte pieces whichever way the operand lies in memory;
//    where k is contiguous there and the 16 bytes are aligned and whole, its
//    load is too, otherwise it is by element.
//  * The next slice's loads are issued before the current one's products.
//  * The matrix instruction gets the operands swapped, so that a lane holds
//    four consecutive columns of one row of the result.
// 64-bit addresses throughout; what lies outside the operands is not read and
// counts as zero.
#include <utility>

#include "grouped_internal.h"

namespace gemm {
namespace grouped {
namespace {

constexpr int TILE = 64, THREADS = 256;
[[maybe_unused]] constexpr int BK = 32;

template <int DT>
struct TypeOf;
template <>
struct TypeOf<GEMM_DTYPE_F32> { typedef float type; };
template <>
struct TypeOf<GEMM_DTYPE_F16> { typedef _Float16 type; };
template <>
struct TypeOf<GEMM_DTYPE_BF16> { typedef __bf16 type; };

template <class T>
struct Operand {
  const T* at;    // element (0, 0) of the tile
  int64_t ld;
  int rows;       // rows (columns of the result) inside the operand, of 64
  int vec;        // k contiguous: 16-byte pieces are aligned
};

// Eight values k0 .. k0 + 7 of one row, of which `left` are inside.
// ACROSS: rows are contiguous in memory, k is `ld` apart.
template <class T, bool ACROSS>
__device__ __forceinline__ void load8(const Operand<T>& o, int row, int64_t k0, int64_t left, T (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (T)0.f;
  if (row >= o.rows || left <= 0) return;
  if constexpr (ACROSS) {
    const T* p = o.at + k0 * o.ld + row;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) v[i] = p[i * o.ld];
  } else {
    const T* p = o.at + row * o.ld + k0;
    if (o.vec && left >= 8) {
      __builtin_memcpy(v, __builtin_assume_aligned(p, 16), 8 * sizeof(T));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) v[i] = p[i];
    }
  }
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// acc[j][i], register e of lane l: row 16i + l%16, column 16j + 4(l/16) + e
// of the wave's 32 x 32 share (row (wave/2), column (wave%2)).
template <int DT, bool AX, bool BX>
__device__ __forceinline__ void tile_sums(const Operand<typename TypeOf<DT>::type>& A,
                                          const Operand<typename TypeOf<DT>::type>& B, int64_t K, f32x4 (&acc)[2][2]) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename TypeOf<DT>::type T;
  constexpr int ROW = BK + 16 / (int)sizeof(T);
  __shared__ __attribute__((aligned(16))) T la[TILE * ROW], lb[TILE * ROW];
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16, wave = tid >> 6;
  // Rows across: a wave takes 64 rows of one k run; otherwise four lanes take
  // one row's 32 k.
  const int ra = AX ? tid % 64 : tid / 4, ka = 8 * (AX ? tid / 64 : tid % 4);
  const int rb = BX ? tid % 64 : tid / 4, kb = 8 * (BX ? tid / 64 : tid % 4);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  T va[8], vb[8];
  load8<T, AX>(A, ra, ka, K - ka, va);
  load8<T, BX>(B, rb, kb, K - kb, vb);
  for (int64_t k0 = 0; k0 < K; k0 += BK) {
    __syncthreads();
    __builtin_memcpy(__builtin_assume_aligned(la + ra * ROW + ka, 16), va, sizeof(va));
    __builtin_memcpy(__builtin_assume_aligned(lb + rb * ROW + kb, 16), vb, sizeof(vb));
    __syncthreads();
    const int64_t next = k0 + BK;
    load8<T, AX>(A, ra, next + ka, K - next - ka, va);
    load8<T, BX>(B, rb, next + kb, K - next - kb, vb);
    const T* pa = la + (32 * (wave / 2) + r) * ROW;
    const T* pb = lb + (32 * (wave % 2) + r) * ROW;
    if constexpr (DT == GEMM_DTYPE_F32) {
      // Lane group q takes k 16h + 4q .. + 3, one in each of four
      // instructions (any order common to both operands will do).
#pragma unroll
      for (int h = 0; h < BK / 16; ++h) {
        f32x4 a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = *(const f32x4*)(pa + 16 * i * ROW + 16 * h + 4 * q);
          b[i] = *(const f32x4*)(pb + 16 * i * ROW + 16 * h + 4 * q);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j][e], a[i][e], acc[j][i], 0, 0, 0);
      }
    } else {
      h16x8_t a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *(const h16x8_t*)(pa + 16 * i * ROW + 8 * q);
        b[i] = *(const h16x8_t*)(pb + 16 * i * ROW + 8 * q);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[j][i] = mfma16<DT == GEMM_DTYPE_BF16>(b[j], a[i], acc[j][i]);
    }
  }
#endif
}

// Calls f(row, column, value) for the lane's results inside rows x cols.
template <class F>
__device__ __forceinline__ void each_result(const f32x4 (&acc)[2][2], int rows, int cols, F&& f) {
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 32 * (wave / 2) + 16 * i + l % 16;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = 32 * (wave % 2) + 16 * j + 4 * (l / 16) + e;
        if (row < rows && col < cols) f(row, col, acc[j][i][e]);
      }
  }
}

// (A grid has at most 2^22 workgroups; they walk over the tiles.)
constexpr int64_t kMostBlocks = 1 << 22;

template <int DT, int CT, bool TRANS>
__global__ void __launch_bounds__(THREADS) matmul_general(MatmulArgs p, int64_t tiles, int tiles_n, int vec_x, int vec_w) {
  typedef typename TypeOf<DT>::type T;
  typedef typename TypeOf<CT>::type C;
  const RowTiles all(p.offsets, p.G, p.T, p.fill, TILE);
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    const RowTile t = all.find((int)(b / tiles_n));
    if (t.rows <= 0) return;  // (`tiles` are the most that offsets can give, in the order of the rows)
    const int n0 = (int)(b % tiles_n) * TILE, cols = p.N - n0 < TILE ? p.N - n0 : TILE;
    const T* X = static_cast<const T*>(p.X) + t.row0 * p.ldx;
    const T* W = static_cast<const T*>(p.W) + (t.g < 0 ? 0 : t.g) * p.stride_w + (TRANS ? n0 * p.ldw : n0);
    f32x4 acc[2][2];
    // (Rows of no group: a sum over no k.)
    tile_sums<DT, false, !TRANS>(Operand<T>{X, p.ldx, t.rows, vec_x}, Operand<T>{W, p.ldw, cols, vec_w}, t.g < 0 ? 0 : p.K,
                                 acc);
    C* Y = static_cast<C*>(p.Y) + t.row0 * p.ldy + n0;
    each_result(acc, t.rows, cols, [&](int row, int col, float v) { Y[row * p.ldy + col] = (C)v; });
  }
}

template <int DT, int CT>
__global__ void __launch_bounds__(THREADS) wgrad_general(WgradArgs p, int64_t tiles, int tiles_k, int tiles_n) {
  typedef typename TypeOf<DT>::type T;
  typedef typename TypeOf<CT>::type C;
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    const int64_t each = (int64_t)tiles_k * tiles_n, in = b % each;
    const int g = (int)(b / each), m0 = (int)(in / tiles_n) * TILE, n0 = (int)(in % tiles_n) * TILE;
    const int rows = p.K - m0 < TILE ? p.K - m0 : TILE, cols = p.N - n0 < TILE ? p.N - n0 : TILE;
    int start, end;
    group_rows(p.offsets, p.T, g, start, end);
    f32x4 acc[2][2];
    tile_sums<DT, true, true>(Operand<T>{static_cast<const T*>(p.X) + start * p.ldx + m0, p.ldx, rows, 0},
                              Operand<T>{static_cast<const T*>(p.dY) + start * p.ldy + n0, p.ldy, cols, 0}, end - start, acc);
    C* W = static_cast<C*>(p.dW) + g * p.stride_w + m0 * p.ldw + n0;
    each_result(acc, rows, cols, [&](int row, int col, float v) {
      C* at = W + row * p.ldw + col;
      v *= p.alpha;
      if (p.beta != 0.f) v = __builtin_fmaf(p.beta, (float)*at, v);
      *at = (C)v;
    });
  }
}

dim3 grid_of(int64_t tiles) { return dim3((unsigned)(tiles < kMostBlocks ? tiles : kMostBlocks)); }

template <int DT, int CT>
hipError_t launch(const MatmulArgs& a, hipStream_t s) {
  const int64_t es = sizeof(typename TypeOf<DT>::type);
  const auto aligned = [&](const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld * es % 16 == 0; };
  const int64_t tiles_n = ((int64_t)a.N + TILE - 1) / TILE, tiles = most_tiles(a.T, a.G, a.fill, TILE) * tiles_n;
  if (tiles <= 0) return hipSuccess;
  const int vx = aligned(a.X, a.ldx), vw = aligned(a.W, a.ldw) && a.stride_w * es % 16 == 0;
  if (a.trans_w)
    hipLaunchKernelGGL((matmul_general<DT, CT, true>), grid_of(tiles), dim3(THREADS), 0, s, a, tiles, (int)tiles_n, vx, vw);
  else
    hipLaunchKernelGGL((matmul_general<DT, CT, false>), grid_of(tiles), dim3(THREADS), 0, s, a, tiles, (int)tiles_n, vx, vw);
  return hipGetLastError();
}

template <int DT, int CT>
hipError_t launch(const WgradArgs& a, hipStream_t s) {
  const int64_t tiles_k = ((int64_t)a.K + TILE - 1) / TILE, tiles_n = ((int64_t)a.N + TILE - 1) / TILE;
  const int64_t tiles = a.G * tiles_k * tiles_n;
  if (tiles <= 0) return hipSuccess;
  hipLaunchKernelGGL((wgrad_general<DT, CT>), grid_of(tiles), dim3(THREADS), 0, s, a, tiles, (int)tiles_k, (int)tiles_n);
  return hipGetLastError();
}

template <class Args>
hipError_t dispatch(int dtype, int c_dtype, const Args& a, hipStream_t s) {
  if (dtype == GEMM_DTYPE_F32) return launch<GEMM_DTYPE_F32, GEMM_DTYPE_F32>(a, s);
  if (dtype == GEMM_DTYPE_F16)
    return c_dtype == GEMM_DTYPE_F32 ? launch<GEMM_DTYPE_F16, GEMM_DTYPE_F32>(a, s) : launch<GEMM_DTYPE_F16, GEMM_DTYPE_F16>(a, s);
  return c_dtype == GEMM_DTYPE_F32 ? launch<GEMM_DTYPE_BF16, GEMM_DTYPE_F32>(a, s) : launch<GEMM_DTYPE_BF16, GEMM_DTYPE_BF16>(a, s);
}

}  // namespace

hipError_t launch_general(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s) { return dispatch(dtype, c_dtype, a, s); }
hipError_t launch_general(int dtype, int c_dtype, const WgradArgs& a, hipStream_t s) { return dispatch(dtype, c_dtype, a, s); }

}  // namespace grouped
}  // namespace gemm

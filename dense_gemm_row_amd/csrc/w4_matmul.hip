// Products of few rows with 4-bit weights (include/gemm_w4.h), dense and
// grouped: Y[t] = X[t] x W^T with
//   W[n][k] = s[n][j] (q[n][k] - z[n][j]),  j = k / group, so that
//   Y[t][n] = sum_j s[n][j] (sum_{k in j} q X[t][k] - z[n][j] sum_{k in j} X[t][k]).
// Bound by the bytes of the codes; every instruction on them counts.
//  * A workgroup of eight waves computes 16 MB rows x 16 NB columns; the waves
//    take spans of SPAN k in turn and their sums are added in wave order
//    through LDS.  There is no other staging: a wave's codes are read straight
//    into operand registers, 16 rows of SPAN / 2 bytes.
//  * The codes of a group lie in a lane's load of group / 8 bytes: lane group q
//    (of four) takes the q-th quarter of the group's k (any order common to
//    both operands will do), a word of 8 codes for each matrix instruction.
//  * A byte 0 .. 15 read as E4M3 is that number times 2^-9 (subnormals and the
//    first exponent are one linear run), so the conversion from E4M3 with the
//    factor 2^9 gives whole numbers in the activations' type, exactly: two
//    masks and a shift, two byte permutes and four conversions for 8 codes.
//  * sum X comes from one more matrix instruction per group's step with ones
//    for weights; it has the layout of the other sums, and all NB blocks of
//    columns share it.  Zero point and scale are two fused operations a value.
#include "grouped_internal.h"
#include "w4_internal.h"

namespace gemm {
namespace w4 {
namespace {

constexpr int WAVES = 8, SPAN = 256;
constexpr int64_t kMostBlocks = 1 << 22;

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Eight codes as eight values of the type, in order.
template <bool BF>
__device__ __forceinline__ u32x4 widen(unsigned word) {
  u32x4 v = {0, 0, 0, 0};
#if defined(__HIP_DEVICE_COMPILE__)
  const unsigned even = word & 0x0f0f0f0fu, odd = (word >> 4) & 0x0f0f0f0fu;
  const unsigned a = __builtin_amdgcn_perm(odd, even, 0x05010400u), b = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  constexpr float up = 512.f;
  if constexpr (BF) {
    v[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, up, false));
    v[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, up, true));
    v[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, up, false));
    v[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, up, true));
  } else {
    v[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, up, false));
    v[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, up, true));
    v[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, up, false));
    v[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, up, true));
  }
#endif
  return v;
}

template <bool BF, int GB, int MB, int NB>
__global__ void __launch_bounds__(64 * WAVES) matmul_few(MatmulArgs p, int64_t tiles, int tiles_n, int vec_x, int vec_s) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef half_t<BF> T;
  constexpr int V = GB / 32;          // words of a lane's load, matrix instructions of a group
  constexpr int GROUPS = SPAN / GB;   // groups of a span
  constexpr int ROWS = 16 * MB, COLS = 16 * NB;
  __shared__ float sums[WAVES][ROWS][COLS];
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ng = (p.K + GB - 1) / GB, padded = (p.K + 31) / 32 * 32;
  const unsigned one = BF ? 0x3f803f80u : 0x3c003c00u;
  const h16x8_t ones = __builtin_bit_cast(h16x8_t, u32x4{one, one, one, one});

  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    grouped::RowTile t;
    if (p.offsets) {
      t = grouped::find_tile(p.offsets, p.G, p.T, p.fill, ROWS, (int)(b / tiles_n));
      if (t.rows <= 0) break;
    } else {
      t.g = 0;
      t.row0 = (int)(b / tiles_n) * ROWS;
      t.rows = p.T - t.row0 < ROWS ? p.T - t.row0 : ROWS;
    }
    const int n0 = (int)(b % tiles_n) * COLS;
    // Rows and columns past the end read the last one's; their results are
    // not stored.
    const T* x[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row = 16 * i + r < t.rows ? 16 * i + r : t.rows - 1;
      x[i] = static_cast<const T*>(p.X) + (t.row0 + row) * p.ldx;
    }
    const int64_t g = t.g < 0 ? 0 : t.g;
    const uint8_t *codes[NB], *zeros[NB];
    const T* scales[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int64_t n = n0 + 16 * j + r < p.N ? n0 + 16 * j + r : p.N - 1;
      codes[j] = p.codes + g * p.stride_q + n * p.ldq;
      scales[j] = static_cast<const T*>(p.scales) + g * p.stride_s + n * p.lds;
      zeros[j] = p.zeros ? p.zeros + g * p.stride_z + n * p.ldz : nullptr;
    }
    f32x4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int K = t.g < 0 ? 0 : p.K;  // (rows of no group: a sum over no k)
    for (int64_t at = (int64_t)wave * SPAN; at < K; at += WAVES * SPAN) {
      const int k0 = (int)at;
      const bool inside = p.K - k0 >= SPAN;
      unsigned w[NB][GROUPS][V];
      float s[NB][GROUPS], z[NB][GROUPS];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int h = 0; h < GROUPS; ++h) {
          int k = k0 + GB * h + 8 * V * q;  // (the lane's piece lies in whole 32 k, all of it there or none)
          if (!inside && k >= padded) k = 0;
          __builtin_memcpy(w[j][h], __builtin_assume_aligned(codes[j] + k / 2, 4 * V), 4 * V);
        }
        if (inside && vec_s) {
          T sv[GROUPS];
          __builtin_memcpy(sv, __builtin_assume_aligned(scales[j] + k0 / GB, sizeof(sv)), sizeof(sv));
          uint8_t zv[GROUPS];
          if (p.zeros) __builtin_memcpy(zv, __builtin_assume_aligned(zeros[j] + k0 / GB, sizeof(zv)), sizeof(zv));
#pragma unroll
          for (int h = 0; h < GROUPS; ++h) {
            s[j][h] = (float)sv[h];
            z[j][h] = p.zeros ? (float)zv[h] : 8.f;
          }
        } else {
#pragma unroll
          for (int h = 0; h < GROUPS; ++h) {
            const int at_group = k0 / GB + h < ng ? k0 / GB + h : ng - 1;
            s[j][h] = (float)scales[j][at_group];
            z[j][h] = p.zeros ? (float)zeros[j][at_group] : 8.f;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < GROUPS; ++h) {
        if (k0 / GB + h >= ng) break;
        f32x4 part[NB][MB], sx[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          sx[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < NB; ++j) part[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int k = k0 + GB * h + 8 * V * q + 8 * v;
          h16x8_t xv[MB];
#pragma unroll
          for (int i = 0; i < MB; ++i) {
            if (inside && vec_x) {
              xv[i] = *reinterpret_cast<const h16x8_t*>(x[i] + k);
            } else {
              T e[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) e[c] = k + c < p.K ? x[i][k + c] : (T)0.f;
              xv[i] = __builtin_bit_cast(h16x8_t, e);
            }
            sx[i] = mfma16<BF>(xv[i], ones, sx[i]);
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const h16x8_t wv = __builtin_bit_cast(h16x8_t, widen<BF>(w[j][h][v]));
#pragma unroll
            for (int i = 0; i < MB; ++i) part[j][i] = mfma16<BF>(xv[i], wv, part[j][i]);
          }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[j][i][e] = __builtin_fmaf(s[j][h], __builtin_fmaf(-z[j][h], sx[i][e], part[j][i][e]), acc[j][i][e]);
      }
    }

    // Register e of lane l: row 16i + 4q + e, column 16j + r.
    __syncthreads();  // (the sums of the tile before have been read)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][16 * i + 4 * q + e][16 * j + r] = acc[j][i][e];
    __syncthreads();
    for (int i = tid; i < ROWS * COLS; i += 64 * WAVES) {
      const int m = i / COLS, n = i % COLS;
      if (m >= t.rows || n0 + n >= p.N) continue;
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < WAVES; ++u) v += sums[u][m][n];
      static_cast<T*>(p.Y)[(t.row0 + m) * p.ldy + n0 + n] = (T)v;
    }
  }
#endif
}

template <bool BF, int GB, int MB, int NB>
hipError_t launch(const MatmulArgs& a, hipStream_t s) {
  constexpr int64_t rows = 16 * MB, cols = 16 * NB, spans = SPAN / GB;
  const int64_t tiles_n = (a.N + cols - 1) / cols;
  const int64_t tiles_m = a.offsets ? grouped::most_tiles(a.T, a.G, a.fill, rows) : (a.T + rows - 1) / rows;
  const int64_t tiles = tiles_m * tiles_n;
  if (tiles <= 0) return hipSuccess;
  const int vec_x = (uintptr_t)a.X % 16 == 0 && a.ldx % 8 == 0;
  // The scales and zero points of a span as one load each.
  const int vec_s = (uintptr_t)a.scales % (2 * spans) == 0 && a.lds % spans == 0 && (a.G <= 1 || a.stride_s % spans == 0) &&
                    (!a.zeros || ((uintptr_t)a.zeros % spans == 0 && a.ldz % spans == 0 && (a.G <= 1 || a.stride_z % spans == 0)));
  hipLaunchKernelGGL((matmul_few<BF, GB, MB, NB>), dim3((unsigned)(tiles < kMostBlocks ? tiles : kMostBlocks)),
                     dim3(64 * WAVES), 0, s, a, tiles, (int)tiles_n, vec_x, vec_s);
  return hipGetLastError();
}

template <bool BF, int GB>
hipError_t by_rows(const MatmulArgs& a, hipStream_t s) {
  // Rows that a tile is likely to have.
  const int64_t rows = a.offsets ? ((int64_t)a.T + a.G - 1) / (a.G > 0 ? a.G : 1) : a.T;
  if (rows <= 16) return launch<BF, GB, 1, 1>(a, s);
  if (rows <= 32) return launch<BF, GB, 2, 1>(a, s);
  return launch<BF, GB, 4, 1>(a, s);
}

template <bool BF>
hipError_t by_group(int group, const MatmulArgs& a, hipStream_t s) {
  if (group == 32) return by_rows<BF, 32>(a, s);
  if (group == 64) return by_rows<BF, 64>(a, s);
  return by_rows<BF, 128>(a, s);
}

}  // namespace

hipError_t launch_matmul(int dtype, int group, const MatmulArgs& a, hipStream_t s) {
  return dtype == GEMM_DTYPE_BF16 ? by_group<true>(group, a, s) : by_group<false>(group, a, s);
}

}  // namespace w4
}  // namespace gemm

// The grouped product for groups of few rows (a decoding step's), 16-bit
// operands of whole 16-byte pieces: bound by the bytes of the weights, so all
// that counts is how many of them are on their way.
//  * A workgroup of four waves computes 16 rows x 64 columns, each wave a
//    quarter of k on its own, without a barrier; the sums are added in order
//    through LDS at the end.
//  * A wave streams slices of 64 k (2 KB of X, 8 KB of W) through four LDS
//    stages of its own with 16-byte LDS-direct copies, three slices ahead of
//    the one it multiplies: 120 KB a CU are on their way.
//    (One row each through 8 of 64 experts of 2048 x 1024: 9.3 us, 3.6 TB/s;
//    22 us on the 128 x 128 tile, which has 64 workgroups there.)
//  * The layouts in LDS are those of the pipelined kernels (grouped_pipe.hip):
//    128-byte rows, for W as it lies k x n with another XOR of the chunks, 2 (k /
//    2 % 2) + 4 (k / 8 % 2), as rows of 64 columns are half as long.
#include "grouped_internal.h"
#include "mx_pipe.h"

namespace gemm {
namespace grouped {
namespace {

using mx::OOB;
using mx::f32x4;
using mx::i32x2;
using mx::i32x4;

constexpr int ROWS = 16, COLS = 64, WAVES = 4, BK = 64;
constexpr int A_STAGE = ROWS * 2 * BK, B_STAGE = COLS * 2 * BK, IA = A_STAGE / 1024, IB = B_STAGE / 1024;
[[maybe_unused]] constexpr int LPS = IA + IB;  // copies of a slice
constexpr int64_t kMostBlocks = 1 << 23;

[[maybe_unused]] __host__ __device__ constexpr int along_swz(int row) { return row / 2 % 8; }
[[maybe_unused]] __host__ __device__ constexpr int across_swz(int k) { return (2 * (k / 2 % 2)) ^ (4 * (k / 8 % 2)); }

template <bool BF, bool ACROSS>
__global__ void __launch_bounds__(64 * WAVES) matmul_few(MatmulArgs p, unsigned tiles, unsigned tiles_n, int c32) {
#if defined(__HIP_DEVICE_COMPILE__)
  // (Stages are arrays of their own: the compiler sees that copies into one do
  // not touch what is read from another.)
  __shared__ __attribute__((aligned(1024))) uint8_t s0[WAVES][A_STAGE + B_STAGE], s1[WAVES][A_STAGE + B_STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[WAVES][A_STAGE + B_STAGE], s3[WAVES][A_STAGE + B_STAGE];
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const RowTiles all(p.offsets, p.G, p.T, p.fill, ROWS);
  // This lane's chunks: of X and (W along k) of W, chunk l % 8 of row 8i + l / 8.
  const int line = l / 8;
  int a_fb[2], b_fb[ACROSS ? 4 : 2];
#pragma unroll
  for (int j = 0; j < 2; ++j) a_fb[j] = 128 * r + 16 * ((4 * j + q) ^ along_swz(r));
#pragma unroll
  for (int i = 0; i < (ACROSS ? 4 : 2); ++i) {
    if constexpr (ACROSS) {
      const int k = 8 * q + r / 4, n = 16 * i + 4 * (r % 4);
      b_fb[i] = 128 * k + 16 * (n / 8 ^ across_swz(k)) + 2 * (n % 8);
    } else {
      b_fb[i] = a_fb[i];  // (columns r of a block, 2 KB a block)
    }
  }

  for (unsigned b = blockIdx.x; b < tiles; b += gridDim.x) {
    const RowTile t = all.find((int)(b / tiles_n));
    if (t.rows <= 0) return;  // (`tiles` are the most that offsets can give, in the order of the rows)
    // (Said to be uniform: the descriptors have to be in scalar registers.)
    const int g = __builtin_amdgcn_readfirstlane(t.g), row0 = __builtin_amdgcn_readfirstlane(t.row0);
    const int rows = __builtin_amdgcn_readfirstlane(t.rows), n0 = __builtin_amdgcn_readfirstlane((int)(b % tiles_n) * COLS);
    const int cols = p.N - n0 < COLS ? p.N - n0 : COLS;
    const int K = g < 0 ? 0 : p.K;  // (rows of no group: a sum over no k)
    const uint16_t* X = static_cast<const uint16_t*>(p.X) + row0 * p.ldx;
    const uint16_t* W = static_cast<const uint16_t*>(p.W) + (g < 0 ? 0 : g) * p.stride_w + (ACROSS ? n0 : n0 * p.ldw);
    const int ldx = (int)p.ldx, ldw = (int)p.ldw;
    // This wave's slices, first ... first + slices - 1.
    const int share = ((K + BK - 1) / BK + WAVES - 1) / WAVES, first = wave * share * BK;
    const int end = K < first + share * BK ? K : first + share * BK, slices = end > first ? (end - first + BK - 1) / BK : 0;
    unsigned a_off[IA], b_off[IB];
    int a_chunk[IA], b_chunk[IB];
#pragma unroll
    for (int i = 0; i < IA; ++i) {
      const int row = 8 * i + line;
      a_chunk[i] = l % 8 ^ along_swz(row);
      a_off[i] = row < rows ? (unsigned)(2 * (row * ldx + 8 * a_chunk[i])) : OOB;
    }
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      const int row = 8 * i + line;
      b_chunk[i] = l % 8 ^ (ACROSS ? across_swz(row) : along_swz(row));
      if constexpr (ACROSS) b_off[i] = 8 * b_chunk[i] < cols ? (unsigned)(2 * (row * ldw + 8 * b_chunk[i])) : OOB;
      else b_off[i] = row < cols ? (unsigned)(2 * (row * ldw + 8 * b_chunk[i])) : OOB;
    }
    // Slice i into a stage; what lies past the wave's k comes as zeros.
    auto copy = [&](int i, uint8_t* stage) __attribute__((always_inline)) {
      const int k0 = first + BK * i, left = end - k0;
      const __amdgpu_buffer_rsrc_t ra = mx::make_rsrc(X + k0, 0x7fffffff);
      const int n = left < BK ? left : BK;
      const __amdgpu_buffer_rsrc_t rb = ACROSS ? mx::make_rsrc(W + (int64_t)k0 * ldw, n > 0 ? 2 * ((n - 1) * ldw + ((cols + 7) & ~7)) : 0)
                                               : mx::make_rsrc(W + k0, 0x7fffffff);
#pragma unroll
      for (int c = 0; c < IB; ++c) {
        const unsigned off = ACROSS || 8 * b_chunk[c] < left ? b_off[c] : OOB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (mx::lds_void*)(stage + A_STAGE + 1024 * c), 16, off, 0, 0, 0);
      }
#pragma unroll
      for (int c = 0; c < IA; ++c) {
        const unsigned off = 8 * a_chunk[c] < left ? a_off[c] : OOB;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (mx::lds_void*)(stage + 1024 * c), 16, off, 0, 0, 0);
      }
    };
    f32x4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Slice i from its stage, once all but the copies of three slices after it
    // have landed; those of the third go where the slice before it was.
    auto slice = [&](int i, const uint8_t* stage, uint8_t* before) __attribute__((always_inline)) {
      static_assert(3 * LPS == 30, "the wait below");
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the slice before has been read
      copy(i + 3, before);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0x4f7e);  // vmcnt(30)
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const h16x8_t x = __builtin_bit_cast(h16x8_t, *(const mx::lds_i32x4*)(stage + a_fb[j]));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          i32x4 w;
          if constexpr (ACROSS) {
            const uint8_t* at = stage + A_STAGE + b_fb[c] + 128 * 32 * j;
            const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx::lds_s16x4*)at));
            const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx::lds_s16x4*)(at + 128 * 4)));
            w = __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
          } else {
            w = *(const mx::lds_i32x4*)(stage + A_STAGE + b_fb[j] + 128 * 16 * c);
          }
          acc[c] = mfma16<BF>(x, __builtin_bit_cast(h16x8_t, w), acc[c]);
        }
      }
    };
    copy(0, s0[wave]);
    copy(1, s1[wave]);
    copy(2, s2[wave]);
    for (int i = 0; i < slices; i += 4) {
      slice(i, s0[wave], s3[wave]);
      slice(i + 1, s1[wave], s0[wave]);
      slice(i + 2, s2[wave], s1[wave]);
      slice(i + 3, s3[wave], s2[wave]);
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // (the copies past the end too: the sums go where they land)

    // Register e of lane l: row 4q + e, column 16j + r.
    float* const sums = reinterpret_cast<float*>(s0);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sums[(wave * ROWS + 4 * q + e) * COLS + 16 * j + r] = acc[j][e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS * COLS / (64 * WAVES); ++i) {
      const int at = i * 64 * WAVES + tid, m = at / COLS, n = at % COLS;
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < WAVES; ++u) v += sums[u * ROWS * COLS + at];
      if (m >= rows || n >= cols) continue;
      const int64_t to = (row0 + m) * p.ldy + n0 + n;
      if (c32) static_cast<float*>(p.Y)[to] = v;
      else static_cast<unsigned short*>(p.Y)[to] = round16<BF>(v);
    }
    __syncthreads();  // (the next tile's copies come where the sums were)
  }
#endif
}

}  // namespace

hipError_t launch_few(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s) {
  const int64_t tiles_n = ((int64_t)a.N + COLS - 1) / COLS, tiles = most_tiles(a.T, a.G, a.fill, ROWS) * tiles_n;
  if (tiles == 0) return hipSuccess;
  const dim3 grid((unsigned)(tiles < kMostBlocks ? tiles : kMostBlocks)), block(64 * WAVES);
  const int c32 = c_dtype == GEMM_DTYPE_F32;
  auto start = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a, (unsigned)tiles, (unsigned)tiles_n, c32);
  };
  if (dtype == GEMM_DTYPE_BF16) a.trans_w ? start(matmul_few<true, false>) : start(matmul_few<true, true>);
  else a.trans_w ? start(matmul_few<false, false>) : start(matmul_few<false, true>);
  return hipGetLastError();
}

}  // namespace grouped
}  // namespace gemm

// Product of two E2M1 (MXFP4) matrices, C = act(alpha A Bt^T + beta C + bias)
// (include/gemm_mx.h), on v_mfma_scale_f32_16x16x128_f8f6f4.
//
// The instruction multiplies 128 k values of 16 rows by 16 columns: lane l
// holds row l%16's 32 values of k block l/16 (16 bytes of codes) and that
// block's scale byte, which is exactly the storage format, so codes and
// scales go from memory to the matrix core without a conversion.  The
// operands are swapped (the result is C^T's block): register i of lane l is
// then C[l%16][4(l/16) + i], four consecutive columns of one row.
#include "mx_internal.h"

namespace gemm {
namespace mx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int FP4 = 4;  // operand format field

__device__ __forceinline__ f32x4 mfma_fp4(i32x4 a, int sa, i32x4 b, int sb, f32x4 c) {
  const i32x8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, FP4, FP4, 0, sa, 0, sb);
}

// Columns n .. n+3 of row m from their sums (n < N; the row has N columns).
template <int DT>
__device__ __forceinline__ void store4(const MatmulArgs& p, int64_t m, int64_t n, f32x4 acc) {
  typedef typename TypeOf<DT>::type T;
  typedef T t4 __attribute__((ext_vector_type(4)));
  T* c = static_cast<T*>(p.C) + m * p.ldc + n;
  const bool whole = n + 4 <= p.N && ((uintptr_t)c & (sizeof(t4) - 1)) == 0;
  if (p.epi.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= p.N) break;
      const float old = p.epi.beta != 0.f ? (float)c[i] : 0.f;
      acc[i] = epi_value(p.epi, acc[i], old, p.epi.bias ? p.epi.bias[n + i] : 0.f);
    }
  }
  if (whole) {
    *reinterpret_cast<t4*>(c) = t4{(T)acc[0], (T)acc[1], (T)acc[2], (T)acc[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) c[i] = (T)acc[i];
  }
}

// A workgroup of W waves computes MT*16 rows x NT*16 columns; the waves
// take turns along k, U instructions' depth (U * 128) each, straight from
// memory, and their sums meet in LDS in wave order.  Rows and columns past
// the matrix repeat its last one and are not stored; blocks past the last
// are zeros.
template <int DT, int MT, int NT, int W, int U>
__global__ void __launch_bounds__(64 * W)
matmul_direct(MatmulArgs p, int tiles_n, int64_t tiles) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  __shared__ __attribute__((aligned(16))) float sums[W][BM][BN];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane % 16, q = lane / 16;
  const int nb = (p.K + BLOCK - 1) / BLOCK;
  const int steps = (nb + 3) / 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile / tiles_n * BM, n0 = tile % tiles_n * BN;
    const uint8_t *ac[MT], *as[MT], *bc[NT], *bs[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int64_t m = m0 + 16 * i + r, row = m < p.M ? m : p.M - 1;
      ac[i] = p.a.codes + row * p.a.ldq;
      as[i] = p.a.scales + row * p.a.lds;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = n0 + 16 * j + r, row = n < p.N ? n : p.N - 1;
      bc[j] = p.b.codes + row * p.b.ldq;
      bs[j] = p.b.scales + row * p.b.lds;
    }
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave * U; s0 < steps; s0 += W * U) {
      i32x4 a[U][MT], b[U][NT];
      int sa[U][MT], sb[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int block = 4 * (s0 + u) + q;
        const bool live = block < nb;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          a[u][i] = live ? *reinterpret_cast<const i32x4*>(ac[i] + (int64_t)block * 16) : i32x4{0, 0, 0, 0};
          sa[u][i] = live ? as[i][block] : 127;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b[u][j] = live ? *reinterpret_cast<const i32x4*>(bc[j] + (int64_t)block * 16) : i32x4{0, 0, 0, 0};
          sb[u][j] = live ? bs[j][block] : 127;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mfma_fp4(b[u][j], sb[u][j], a[u][i], sa[u][i], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4*>(&sums[wave][16 * i + r][16 * j + 4 * q]) = acc[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < BM * BN / 4; e += 64 * W) {
      const int m = e / (BN / 4), n = e % (BN / 4) * 4;
      f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][m][n]);
#pragma unroll
      for (int w = 1; w < W; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][m][n]);
      if (m0 + m < p.M && n0 + n < p.N) store4<DT>(p, m0 + m, n0 + n, v);
    }
    __syncthreads();
  }
}

template <int DT, int MT, int NT, int W, int U>
hipError_t launch_direct(const MatmulArgs& a, hipStream_t stream) {
  const int tiles_n = (a.N + 16 * NT - 1) / (16 * NT);
  const int64_t tiles = (int64_t)tiles_n * ((a.M + 16 * MT - 1) / (16 * MT));
  const int64_t most = 1 << 22;  // work-items of a grid: below 2^32
  hipLaunchKernelGGL((matmul_direct<DT, MT, NT, W, U>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(64 * W), 0,
                     stream, a, tiles_n, tiles);
  return hipGetLastError();
}

template <int DT>
hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 16) return launch_direct<DT, 1, 1, 8, 4>(a, stream);
  return launch_direct<DT, 4, 4, 4, 1>(a, stream);
}

}  // namespace

hipError_t launch_matmul(int c_dtype, const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  return c_dtype == GEMM_DTYPE_F32   ? launch<GEMM_DTYPE_F32>(a, stream)
         : c_dtype == GEMM_DTYPE_F16 ? launch<GEMM_DTYPE_F16>(a, stream)
                                     : launch<GEMM_DTYPE_BF16>(a, stream);
}

}  // namespace mx
}  // namespace gemm

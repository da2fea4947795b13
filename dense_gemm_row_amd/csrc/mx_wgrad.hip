// Weight gradient from an 8-bit activation checkpoint, dW = alpha X^T dY +
// beta dW (include/gemm_mx.h): a product summed over tokens, of the E4M3
// codes of X^T (F x T, blocks of 32 tokens) with dY (T x N, row-major).
//
// The bfloat16 matrix instruction takes both operands exactly.  A code is
// four significant bits times a power of two, so v_cvt_scalef32_pk_bf16_fp8
// (code and factor in, bfloat16 out) rounds nothing above bfloat16's
// subnormals.  A binary16 dY is the sum of two bfloat16 terms (8 + 3
// significant bits), an FP32 one of three (8 + 8 + 8), each a truncation of
// what the terms before it left, so the differences are exact; every term
// is one more matrix instruction on the same codes.
#include "mx_internal.h"

namespace gemm {
namespace mx {
namespace {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Eight codes (tokens in order) of one block -> eight bfloat16 values.
__device__ __forceinline__ u32x4 decode8(u32x2 w, float factor) {
  u32x4 v;
  v[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], factor, false));
  v[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], factor, true));
  v[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], factor, false));
  v[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], factor, true));
  return v;
}

// bfloat16 terms of a value of type YT.
template <int YT>
constexpr int kTerms = YT == GEMM_DTYPE_BF16 ? 1 : YT == GEMM_DTYPE_F16 ? 2 : 3;

// The terms' bit patterns, largest first.  Infinities and NaN: the first
// term alone (rounded, which keeps a NaN a NaN).
template <int YT>
__device__ __forceinline__ void split_terms(float x, unsigned short (&t)[kTerms<YT>]) {
  if constexpr (YT == GEMM_DTYPE_BF16) {
    t[0] = (unsigned short)(__builtin_bit_cast(unsigned, x) >> 16);
  } else {
    const unsigned bits = __builtin_bit_cast(unsigned, x);
    const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
    float left = x;
#pragma unroll
    for (int k = 0; k < kTerms<YT>; ++k) {
      const unsigned top = __builtin_bit_cast(unsigned, left) & 0xffff0000u;
      t[k] = (unsigned short)(top >> 16);
      left -= __builtin_bit_cast(float, top);
    }
    if (!finite) {
      t[0] = round16<true>(x);
#pragma unroll
      for (int k = 1; k < kTerms<YT>; ++k) t[k] = 0;
    }
  }
}

template <int DT>
__device__ __forceinline__ float read_as_float(const void* p, int64_t i) {
  return (float)static_cast<const typename TypeOf<DT>::type*>(p)[i];
}

// dW[f][n .. n+3] from its sums.
template <int DT>
__device__ __forceinline__ void store4(const WgradArgs& p, int64_t f, int64_t n, f32x4 acc) {
  typedef typename TypeOf<DT>::type T;
  typedef T t4 __attribute__((ext_vector_type(4)));
  T* c = static_cast<T*>(p.dW) + f * p.ldw + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] *= p.alpha;
    if (p.beta != 0.f && n + i < p.N) acc[i] = __builtin_fmaf(p.beta, (float)c[i], acc[i]);
  }
  if (n + 4 <= p.N && ((uintptr_t)c & (sizeof(t4) - 1)) == 0) {
    *reinterpret_cast<t4*>(c) = t4{(T)acc[0], (T)acc[1], (T)acc[2], (T)acc[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) c[i] = (T)acc[i];
  }
}

// The general kernel: any alignment of dY, every type.  A workgroup of four
// waves computes 64 features x 64 columns, 32 tokens (one block of the
// codes) at a time through LDS: the codes' values token-contiguous, dY's
// terms transposed to token-contiguous while they are staged.
template <int YT, int CT>
__global__ void __launch_bounds__(256)
wgrad_general(WgradArgs p, int tiles_n, int64_t tiles) {
  constexpr int NT = kTerms<YT>;
  constexpr int LD = 40;  // 32 tokens and padding: 80-byte rows spread the banks
  __shared__ __attribute__((aligned(16))) unsigned short xs[64][LD], ys[NT][64][LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wf = (wave / 2) * 32, wn = (wave % 2) * 32;
  const int r = lane % 16, q = lane / 16;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t f0 = tile / tiles_n * 64, n0 = tile % tiles_n * 64;
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int xf = tid / 4, xt = tid % 4 * 8;  // staging: a feature's 8 tokens
    const int yn = tid % 64, yt = tid / 64 * 8;  // a column's 8 tokens
    for (int64_t t0 = 0; t0 < p.T; t0 += BLOCK) {
      u32x4 xv = {0u, 0u, 0u, 0u};
      if (f0 + xf < p.F) {
        const int64_t f = f0 + xf;
        const u32x2 w = *reinterpret_cast<const u32x2*>(p.x.codes + f * p.x.ldq + t0 + xt);
        xv = decode8(w, scale_float(p.x.scales[f * p.x.lds + t0 / BLOCK]));
      }
      *reinterpret_cast<u32x4*>(&xs[xf][xt]) = xv;
      unsigned short terms[8][NT];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t t = t0 + yt + i, n = n0 + yn;
        const bool in = t < p.T && n < p.N;
        split_terms<YT>(in ? read_as_float<YT>(p.dY, t * p.ldy + n) : 0.f, terms[i]);
      }
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = terms[2 * i][k] | ((unsigned)terms[2 * i + 1][k] << 16);
        *reinterpret_cast<u32x4*>(&ys[k][yn][yt]) = v;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        h16x8_t xa[2], yb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          xa[i] = *reinterpret_cast<const h16x8_t*>(&xs[wf + 16 * i + r][8 * q]);
          yb[i] = *reinterpret_cast<const h16x8_t*>(&ys[k][wn + 16 * i + r][8 * q]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma16<true>(yb[j], xa[i], acc[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t f = f0 + wf + 16 * i + r, n = n0 + wn + 16 * j + 4 * q;
        if (f < p.F && n < p.N) store4<CT>(p, f, n, acc[i][j]);
      }
  }
}

template <int YT, int CT>
hipError_t launch(const WgradArgs& a, hipStream_t stream) {
  const int tiles_n = (a.N + 63) / 64;
  const int64_t tiles = (int64_t)tiles_n * ((a.F + 63) / 64);
  const int64_t most = 1 << 22;  // work-items of a grid: below 2^32
  hipLaunchKernelGGL((wgrad_general<YT, CT>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, stream, a,
                     tiles_n, tiles);
  return hipGetLastError();
}

template <int YT>
hipError_t launch(int c_dtype, const WgradArgs& a, hipStream_t stream) {
  return c_dtype == GEMM_DTYPE_F32   ? launch<YT, GEMM_DTYPE_F32>(a, stream)
         : c_dtype == GEMM_DTYPE_F16 ? launch<YT, GEMM_DTYPE_F16>(a, stream)
                                     : launch<YT, GEMM_DTYPE_BF16>(a, stream);
}

}  // namespace

int wgrad_splits(int y_dtype, int64_t T, int64_t F, int64_t N, int* chunk) {
  *chunk = (int)T;
  return 1;
}

hipError_t launch_wgrad(int y_dtype, int c_dtype, const WgradArgs& a, hipStream_t stream) {
  if (a.F <= 0 || a.N <= 0) return hipSuccess;
  return y_dtype == GEMM_DTYPE_F32   ? launch<GEMM_DTYPE_F32>(c_dtype, a, stream)
         : y_dtype == GEMM_DTYPE_F16 ? launch<GEMM_DTYPE_F16>(c_dtype, a, stream)
                                     : launch<GEMM_DTYPE_BF16>(c_dtype, a, stream);
}

}  // namespace mx
}  // namespace gemm

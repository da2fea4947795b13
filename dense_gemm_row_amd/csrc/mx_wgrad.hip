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
#include "mx_pipe.h"

namespace gemm {
namespace mx {
namespace {

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

// dY as bfloat16 terms: plane k of `terms` holds term k of every value, T
// rows of `ld` columns (N rounded up to 8; the rest zeros).
template <int YT>
__global__ void __launch_bounds__(256)
split_planes(const void* dY, int64_t ldy, int64_t T, int N, int groups, unsigned short* out, int64_t plane) {
  constexpr int NT = kTerms<YT>;
  const int64_t total = T * groups;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / groups;
    const int g = (int)(i - t * groups);
    unsigned short terms[8][NT];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = 8 * g + e;
      split_terms<YT>(n < N ? read_as_float<YT>(dY, t * ldy + n) : 0.f, terms[e]);
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = terms[2 * e][k] | ((unsigned)terms[2 * e + 1][k] << 16);
      *reinterpret_cast<u32x4*>(out + k * plane + (t * groups + g) * 8) = v;
    }
  }
}

// dW = alpha * (sum over splits of partial) + beta * dW, added in order;
// partial rows of `ld` (a multiple of 4) columns, four a thread.
template <int CT>
__global__ void __launch_bounds__(256)
reduce_partials(const float* partial, int64_t ld, int64_t stride, int splits, void* dW, int64_t ldw, int64_t F, int N,
                float alpha, float beta) {
  typedef typename TypeOf<CT>::type T;
  typedef T t4 __attribute__((ext_vector_type(4)));
  const int64_t quads = ld / 4, total = F * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t f = i / quads;
    const int n = 4 * (int)(i - f * quads);
    const float* src = partial + f * ld + n;
    f32x4 v = *reinterpret_cast<const f32x4*>(src);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(src + s * stride);
    T* c = static_cast<T*>(dW) + f * ldw + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] *= alpha;
      if (beta != 0.f && n + e < N) v[e] = __builtin_fmaf(beta, (float)c[e], v[e]);
    }
    if (n + 4 <= N && ((uintptr_t)c & (sizeof(t4) - 1)) == 0) {
      *reinterpret_cast<t4*>(c) = t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) c[e] = (T)v[e];
    }
  }
}

template <int CT>
hipError_t launch_tile(int tile, const WgradPipeArgs& a, int splits, hipStream_t stream) {
  return tile == 256 ? launch_wgrad_pipe<CT, 256>(a, splits, stream) : launch_wgrad_pipe<CT, 128>(a, splits, stream);
}

template <int YT, int CT>
hipError_t launch_planned(const WgradArgs& a, const WgradPlan& w, hipStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  WgradPipeArgs p{a.x, static_cast<const uint16_t*>(a.dY), a.ldy, 0, a.dW, a.ldw, 0, a.T, a.F, a.N, 1, w.chunk, a.alpha, a.beta};
  if (w.planes > 0) {
    const int groups = (a.N + 7) / 8;
    p.y = reinterpret_cast<uint16_t*>(ws);
    p.ldy = 8 * (int64_t)groups;
    p.plane = p.ldy * a.T;
    p.terms = kTerms<YT>;
    const int64_t wgs = ((int64_t)a.T * groups + 255) / 256;
    hipLaunchKernelGGL((split_planes<YT>), dim3((unsigned)(wgs < 8192 ? wgs : 8192)), dim3(256), 0, stream, a.dY, a.ldy,
                       (int64_t)a.T, a.N, groups, reinterpret_cast<unsigned short*>(ws), p.plane);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (w.splits <= 1) return launch_tile<CT>(w.tile, p, 1, stream);
  float* partial = reinterpret_cast<float*>(ws + w.planes);
  p.C = partial;
  p.ldc = ((int64_t)a.N + 3) / 4 * 4;
  p.c_stride = p.ldc * a.F;
  p.alpha = 1.f;
  p.beta = 0.f;
  const hipError_t e = launch_tile<GEMM_DTYPE_F32>(w.tile, p, w.splits, stream);
  if (e != hipSuccess) return e;
  const int64_t wgs = (p.c_stride / 4 + 255) / 256;
  hipLaunchKernelGGL((reduce_partials<CT>), dim3((unsigned)(wgs < 8192 ? wgs : 8192)), dim3(256), 0, stream, partial, p.ldc,
                     p.c_stride, w.splits, a.dW, a.ldw, (int64_t)a.F, a.N, a.alpha, a.beta);
  return hipGetLastError();
}

template <int YT, int CT>
hipError_t launch_general(const WgradArgs& a, hipStream_t stream) {
  const int tiles_n = (int)ceil_div(a.N, 64);
  const int64_t tiles = tiles_n * ceil_div(a.F, 64);
  const int64_t most = 1 << 22;  // work-items of a grid: below 2^32
  hipLaunchKernelGGL((wgrad_general<YT, CT>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, stream, a,
                     tiles_n, tiles);
  return hipGetLastError();
}

template <int YT, int CT>
hipError_t launch(const WgradArgs& a, hipStream_t stream) {
  const WgradPlan w = wgrad_plan(YT, a.T, a.F, a.N);
  const bool room = w.bytes() == 0 || (a.workspace && a.workspace_bytes >= w.bytes());
  // What the pipelined kernel takes: scales in 4-byte words, a tile's rows
  // within 31 bits, dY's rows (where they are read as they are) 16-byte
  // aligned.
  const int64_t far = (int64_t)0x7fffffff / 256 - 4096;
  const bool aligned = w.planes > 0 || ((uintptr_t)a.dY % 16 == 0 && a.ldy % 8 == 0);
  if (w.tile == 0 || !room || !aligned || (uintptr_t)a.x.scales % 4 != 0 || a.x.lds % 4 != 0 || a.x.ldq >= far ||
      a.x.lds >= far || a.N >= far || (w.planes == 0 && a.ldy >= far) || a.ldw >= far / 4)
    return launch_general<YT, CT>(a, stream);
  return launch_planned<YT, CT>(a, w, stream);
}

template <int YT>
hipError_t launch(int c_dtype, const WgradArgs& a, hipStream_t stream) {
  return c_dtype == GEMM_DTYPE_F32   ? launch<YT, GEMM_DTYPE_F32>(a, stream)
         : c_dtype == GEMM_DTYPE_F16 ? launch<YT, GEMM_DTYPE_F16>(a, stream)
                                     : launch<YT, GEMM_DTYPE_BF16>(a, stream);
}

}  // namespace

// The pipelined kernel's plan: the tile and the number of token chunks of
// the least modelled time.  Microseconds on MI355X, measured with the card
// full: a slice (64 tokens) of a 256 x 256 tile 1.2 on an idle card to 1.7
// on a full one, of a 128 x 128 tile 0.56 for each that shares a CU; a launch 4; the
// partial sums, written and read, 8 TB/s.  (8192 tokens, 4096 x 4096: 214 us
// on one 256 x 256 tile a CU, 288 on 128 x 128 ones.  16384 tokens, 1024 x
// 1024, on 128 x 128 tiles: 152 us in one chunk, 57 in the 4 that the model
// picks, 51 in 8.  It prices those too high: two workgroups on a CU overlap,
// and it charges each the whole slice.)
WgradPlan wgrad_plan(int y_dtype, int64_t T, int64_t F, int64_t N) {
  WgradPlan best;
  const int64_t cap = (int64_t)1 << 23;  // workgroups of a grid, and columns within a tile's 31 bits
  // One block of tokens or less: the general kernel's one launch (16 tokens,
  // 1024 x 1024: 4.8 us against 7.2).
  if (T <= BLOCK || F <= 0 || N <= 0 || N >= cap || F >= cap * 128) return best;
  const int terms = y_dtype == GEMM_DTYPE_BF16 ? 1 : y_dtype == GEMM_DTYPE_F16 ? 2 : 3;
  const double plane = (double)F * (double)((N + 3) / 4 * 16);
  double least = 1e30;
  for (int tile = 128; tile <= 256; tile += 128) {
    const int64_t tiles = ((F + tile - 1) / tile) * ((N + tile - 1) / tile);
    if (tiles >= cap) continue;
    for (int s = 1; s <= 32; ++s) {
      if (s > 1 && (tiles * s > 1024 || plane * s > (double)(1 << 30))) break;
      const int64_t chunk = ((T + s - 1) / s + 127) / 128 * 128;
      if ((T + chunk - 1) / chunk != s) continue;  // fewer chunks than s: seen already
      const double slices = (double)(chunk / 64) * terms;
      const double wgs = (double)(tiles * s), per_cu = (double)((tiles * s + 255) / 256);
      const double slice = tile == 256 ? 1.2 + 0.5 * (wgs < 256 ? wgs / 256 : 1.) : 0.56;
      const double us = 4 + per_cu * slices * slice + (s > 1 ? 4 + 2 * plane * s / 8e6 : 0.);
      if (us < least) {
        least = us;
        best.tile = tile;
        best.splits = s;
        best.chunk = (int)(chunk > 0x7fffff80 ? 0x7fffff80 : chunk);
      }
    }
  }
  if (best.tile == 0) return best;
  if (terms > 1 || N % 8 != 0) best.planes = terms * T * ((N + 7) / 8) * 16;
  if (best.splits > 1) best.partials = (int64_t)best.splits * F * ((N + 3) / 4) * 16;
  return best;
}

hipError_t launch_wgrad(int y_dtype, int c_dtype, const WgradArgs& a, hipStream_t stream) {
  if (a.F <= 0 || a.N <= 0) return hipSuccess;
  return y_dtype == GEMM_DTYPE_F32   ? launch<GEMM_DTYPE_F32>(c_dtype, a, stream)
         : y_dtype == GEMM_DTYPE_F16 ? launch<GEMM_DTYPE_F16>(c_dtype, a, stream)
                                     : launch<GEMM_DTYPE_BF16>(c_dtype, a, stream);
}

}  // namespace mx
}  // namespace gemm

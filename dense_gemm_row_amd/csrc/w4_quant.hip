// 4-bit weights with group scales: quantisation and back (include/gemm_w4.h).
//
// A code is the whole number nearest to w / s.  The quotient in FP32 can fall
// on a midpoint that the exact one only lies next to, so it is taken as a
// guess (within one of the result) and decided by the exact products: with t
// the guess, w - (t +- 1/2) s in one fused operation has the exact sign ((t +-
// 1/2) s has at most 5 + 11 significant bits, and the one rounding keeps the
// sign).
#include "w4_internal.h"

namespace gemm {
namespace w4 {
namespace {

constexpr int THREADS = 256;
constexpr int64_t kMostBlocks = 1 << 22;  // (kernels walk on from there)

template <int DT>
struct TypeOf;
template <>
struct TypeOf<GEMM_DTYPE_F32> { typedef float type; };
template <>
struct TypeOf<GEMM_DTYPE_F16> { typedef _Float16 type; };
template <>
struct TypeOf<GEMM_DTYPE_BF16> { typedef __bf16 type; };

// The whole number nearest to w / s, ties to even, for s > 0; `inv` is about
// 1 / s.  Beyond +-32 it is cut off (callers clamp to less).
__device__ __forceinline__ float nearest(float w, float s, float inv) {
  float t = __builtin_rintf(__builtin_fminf(__builtin_fmaxf(w * inv, -32.f), 32.f));
  const float up = __builtin_fmaf(-(t + 0.5f), s, w), down = __builtin_fmaf(-(t - 0.5f), s, w);
  const bool odd = ((int)t & 1) != 0;
  if (up > 0.f || (up == 0.f && odd)) t += 1.f;
  else if (down < 0.f || (down == 0.f && odd)) t -= 1.f;
  return t;
}

// A group's scale (as its type's value) and zero point, from its least and
// greatest value and whether all of it is finite.
template <class S>
struct GroupScale {
  S s;
  float value, up, inv, zero;  // (value * up and 1 / it are normal numbers)
  __device__ __forceinline__ GroupScale(float lo, float hi, bool finite, bool zeros) {
    const float most = sizeof(S) == 2 && (float)(S)65536.f != 65536.f ? 65504.f : 0x1.fep127f;
    float x;
    if (zeros) {
      lo = __builtin_fminf(lo, 0.f);
      hi = __builtin_fmaxf(hi, 0.f);
      x = (hi - lo) / 15.f;
    } else {
      x = __builtin_fmaxf(hi, -lo) / 7.f;
    }
    s = (S)__builtin_fminf(x, most);
    value = (float)s;
    // The reciprocal of a subnormal scale may be infinite: a small scale and
    // its values, at most some 15 such scales, are taken 2^64 times larger.
    up = value < 0x1p-60f ? 0x1p64f : 1.f;
    inv = value > 0.f ? 1.f / (value * up) : 0.f;
    zero = zeros ? 0.f : 8.f;
    if (zeros && value > 0.f) zero = __builtin_fminf(__builtin_fmaxf(nearest(-lo * up, value * up, inv), 0.f), 15.f);
    if (!finite) {
      s = (S)__builtin_nanf("");
      value = 0.f;
      zero = 0.f;
    }
  }
  __device__ __forceinline__ unsigned code(float w) const {
    if (!(value > 0.f)) return (unsigned)zero;
    return (unsigned)__builtin_fminf(__builtin_fmaxf(nearest(w * up, value * up, inv) + zero, 0.f), 15.f);
  }
};

template <class T>
__device__ __forceinline__ bool is_finite(T x) {
  return __builtin_fabsf((float)x) < __builtin_inff();  // (false for NaN)
}

// Along rows (X is N x K): GB / 8 lanes take a group, 8 values each.  Bound
// by HBM.
template <class T, class S, int GB>
__global__ void __launch_bounds__(THREADS) quantize_rows(QuantArgs p, int64_t pieces, int per_row, int vec) {
  constexpr int LANES = GB / 8;
  for (int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x; at < pieces; at += (int64_t)gridDim.x * THREADS) {
    // (`pieces` is a multiple of LANES, so a group's lanes run together.)
    const int64_t row = at / per_row;
    const int k0 = 8 * (int)(at % per_row), left = p.K - k0;
    const T* x = static_cast<const T*>(p.X) + row * p.ldx + k0;
    T v[8];
    if (vec && left >= 8) {
      __builtin_memcpy(v, __builtin_assume_aligned(x, 16), sizeof(v));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? x[i] : (T)0.f;
    }
    float lo = 0.f, hi = 0.f;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = __builtin_fminf(lo, (float)v[i]);
      hi = __builtin_fmaxf(hi, (float)v[i]);
      bad |= !is_finite(v[i]);
    }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) {
      lo = __builtin_fminf(lo, __shfl_xor(lo, d));
      hi = __builtin_fmaxf(hi, __shfl_xor(hi, d));
      bad |= __shfl_xor(bad, d);
    }
    const GroupScale<S> g(lo, hi, !bad, p.zeros != nullptr);
    unsigned word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= g.code((float)v[i]) << (4 * i);
    if (k0 < (p.K + 31) / 32 * 32) *reinterpret_cast<unsigned*>(p.codes + row * p.ldq + k0 / 2) = word;
    if (k0 % GB == 0) {
      static_cast<S*>(p.scales)[row * p.lds + k0 / GB] = g.s;
      if (p.zeros) p.zeros[row * p.ldz + k0 / GB] = (uint8_t)g.zero;
    }
  }
}

// Down columns (X is K x N, the codes are its transpose's): a lane takes one
// group of one column, so that a wave reads whole 64-column pieces of X's
// rows; its GB / 2 code bytes are whole 16-byte pieces of its output row.
template <class T, class S, int GB>
__global__ void __launch_bounds__(THREADS) quantize_cols(QuantArgs p, int64_t blocks, int tiles_n) {
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t n = (int64_t)(b % tiles_n) * 64 + threadIdx.x % 64;
    const int64_t j = b / tiles_n * (THREADS / 64) + threadIdx.x / 64, k0 = j * GB;
    if (n >= p.N || k0 >= p.K) continue;
    const int left = p.K - k0 < GB ? (int)(p.K - k0) : GB;
    const T* x = static_cast<const T*>(p.X) + k0 * p.ldx + n;
    T v[GB];
    if (left == GB) {
#pragma unroll
      for (int i = 0; i < GB; ++i) v[i] = x[i * p.ldx];
    } else {
#pragma unroll
      for (int i = 0; i < GB; ++i) v[i] = i < left ? x[i * p.ldx] : (T)0.f;
    }
    float lo = 0.f, hi = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < GB; ++i) {
      lo = __builtin_fminf(lo, (float)v[i]);
      hi = __builtin_fmaxf(hi, (float)v[i]);
      finite = finite && is_finite(v[i]);
    }
    const GroupScale<S> g(lo, hi, finite, p.zeros != nullptr);
    uint8_t* out = p.codes + n * p.ldq + k0 / 2;
#pragma unroll
    for (int c = 0; c < GB / 32; ++c) {
      uint4 w;
      unsigned* words = reinterpret_cast<unsigned*>(&w);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        words[h] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) words[h] |= g.code((float)v[32 * c + 8 * h + i]) << (4 * i);
      }
      if (32 * c < left) *reinterpret_cast<uint4*>(out + 16 * c) = w;
    }
    static_cast<S*>(p.scales)[n * p.lds + j] = g.s;
    if (p.zeros) p.zeros[n * p.ldz + j] = (uint8_t)g.zero;
  }
}

// The values of 8 codes a lane.  s (q - z) has at most 11 + 5 bits, exact in
// FP32, and is rounded once to a 16-bit type.
template <class T, class S>
__global__ void __launch_bounds__(THREADS) dequantize_rows(DequantArgs p, int64_t pieces, int per_row, int group, int vec) {
  const int64_t g = blockIdx.y;
  const uint8_t* codes = p.codes + g * p.stride_q;
  const S* scales = static_cast<const S*>(p.scales) + g * p.stride_s;
  const uint8_t* zeros = p.zeros ? p.zeros + g * p.stride_z : nullptr;
  T* X = static_cast<T*>(p.X) + g * p.stride_x;
  for (int64_t at = (int64_t)blockIdx.x * THREADS + threadIdx.x; at < pieces; at += (int64_t)gridDim.x * THREADS) {
    const int64_t row = at / per_row;
    const int k0 = 8 * (int)(at % per_row), left = p.K - k0;
    const unsigned word = *reinterpret_cast<const unsigned*>(codes + row * p.ldq + k0 / 2);
    const float s = (float)scales[row * p.lds + k0 / group];
    const float z = zeros ? (float)zeros[row * p.ldz + k0 / group] : 8.f;
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)(s * ((float)(word >> (4 * i) & 15) - z));
    T* x = X + row * p.ldx + k0;
    if (vec && left >= 8) {
      __builtin_memcpy(__builtin_assume_aligned(x, 16), v, sizeof(v));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) x[i] = v[i];
    }
  }
}

unsigned blocks_for(int64_t pieces) {
  const int64_t n = (pieces + THREADS - 1) / THREADS;
  return (unsigned)(n < kMostBlocks ? n : kMostBlocks);
}

template <class T, class S, int GB>
hipError_t quantize(bool trans, const QuantArgs& a, hipStream_t s) {
  if (trans) {
    const int64_t tiles_n = ((int64_t)a.N + 63) / 64;
    const int64_t blocks = tiles_n * ((groups_of(a.K, GB) + THREADS / 64 - 1) / (THREADS / 64));
    hipLaunchKernelGGL((quantize_cols<T, S, GB>), dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3(THREADS),
                       0, s, a, blocks, (int)tiles_n);
  } else {
    const int per_row = (int)(groups_of(a.K, GB) * (GB / 8));
    const int vec = (uintptr_t)a.X % 16 == 0 && a.ldx * (int64_t)sizeof(T) % 16 == 0;
    const int64_t pieces = (int64_t)a.N * per_row;
    hipLaunchKernelGGL((quantize_rows<T, S, GB>), dim3(blocks_for(pieces)), dim3(THREADS), 0, s, a, pieces, per_row, vec);
  }
  return hipGetLastError();
}

template <class T, class S>
hipError_t quantize(bool trans, int group, const QuantArgs& a, hipStream_t s) {
  if (group == 32) return quantize<T, S, 32>(trans, a, s);
  if (group == 64) return quantize<T, S, 64>(trans, a, s);
  return quantize<T, S, 128>(trans, a, s);
}

template <class T, class S>
hipError_t dequantize(int group, int G, const DequantArgs& a, hipStream_t s) {
  const int per_row = (int)(((int64_t)a.K + 7) / 8);
  const int vec = (uintptr_t)a.X % 16 == 0 && a.ldx * (int64_t)sizeof(T) % 16 == 0 && a.stride_x * (int64_t)sizeof(T) % 16 == 0;
  const int64_t pieces = (int64_t)a.N * per_row;
  hipLaunchKernelGGL((dequantize_rows<T, S>), dim3(blocks_for(pieces), (unsigned)G), dim3(THREADS), 0, s, a, pieces, per_row,
                     group, vec);
  return hipGetLastError();
}

// f(value of the type, value of the scales' type)
template <class F>
hipError_t by_types(int dtype, int s_dtype, F&& f) {
  const bool sb = s_dtype == GEMM_DTYPE_BF16;
  if (dtype == GEMM_DTYPE_F32) return sb ? f(float(), __bf16()) : f(float(), _Float16());
  if (dtype == GEMM_DTYPE_F16) return sb ? f(_Float16(), __bf16()) : f(_Float16(), _Float16());
  return sb ? f(__bf16(), __bf16()) : f(__bf16(), _Float16());
}

}  // namespace

hipError_t launch_quantize(int dtype, int s_dtype, bool trans, int group, const QuantArgs& a, hipStream_t s) {
  if (a.N == 0 || a.K == 0) return hipSuccess;
  return by_types(dtype, s_dtype, [&](auto t, auto u) { return quantize<decltype(t), decltype(u)>(trans, group, a, s); });
}

hipError_t launch_dequantize(int dtype, int s_dtype, int group, int G, const DequantArgs& a, hipStream_t s) {
  if (a.N == 0 || a.K == 0 || G == 0) return hipSuccess;
  return by_types(dtype, s_dtype, [&](auto t, auto u) { return dequantize<decltype(t), decltype(u)>(group, G, a, s); });
}

}  // namespace w4
}  // namespace gemm

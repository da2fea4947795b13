// 4-bit weights with group scales: quantisation and back (include/gemm_w4.h).
//
// A code is the whole number nearest to w / s.  The quotient in FP32 can fall
// on a midpoint that the exact one only lies next to, so it is taken as a
// guess t, within one of the result, and decided by w - t s, which one fused
// operation gives exactly: it is a multiple of w's last place and, as t is off
// by at most 1/2 + 2^-18, no larger than w (t = 0: w itself).  Above s / 2, or
// at it with t odd, the result is one further.
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

// The whole number nearest to w / s, ties to even, for s > 0; `inv` is 1 / s,
// `half` s / 2 and `above` the next number up.  (Far beyond the codes, where a
// scale is its type's largest, any number of w's sign: callers clamp.)
__device__ __forceinline__ int nearest(float w, float s, float inv, float half, float above) {
  const float t = __builtin_rintf(w * inv), d = __builtin_fmaf(-t, s, w);
  const int i = (int)__builtin_fminf(__builtin_fmaxf(t, -64.f), 64.f);
  const int one = (__builtin_bit_cast(int, d) >> 31) | 1;  // (d's sign)
  return __builtin_fabsf(d) >= (i & 1 ? half : above) ? i + one : i;
}

// A group's scale (as its type's value) and zero point, from its least and
// greatest value and whether all of it is finite.
template <class S>
struct GroupScale {
  S s;
  float value, up, inv, half, above;  // (up: such that the others are normal numbers)
  int zero;
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
    const float scaled = value * up;
    inv = value > 0.f ? 1.f / scaled : 0.f;
    // (A scale of 0: no value is past the half, all codes are the zero point.)
    half = value > 0.f ? 0.5f * scaled : __builtin_inff();
    above = value > 0.f ? __builtin_bit_cast(float, __builtin_bit_cast(unsigned, half) + 1) : __builtin_inff();
    zero = zeros ? 0 : 8;
    if (zeros && value > 0.f) zero = cut(nearest(-lo * up, scaled, inv, half, above));
    if (!finite) {
      s = (S)__builtin_nanf("");
      value = inv = 0.f;
      half = above = __builtin_nanf("");  // (nothing compares with it)
      zero = 0;
    }
  }
  __device__ __forceinline__ static int cut(int i) { return i < 0 ? 0 : i > 15 ? 15 : i; }
  __device__ __forceinline__ unsigned code(float w) const {
    return (unsigned)cut(nearest(w * up, value * up, inv, half, above) + zero);
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

// Down columns (X is K x N, the codes are its transpose's): a lane takes 32 k
// of four columns, 16 lanes 64 columns, GB / 32 groups of 16 lanes a scale's k
// (a wave 128).  So a wave reads whole 128-byte pieces of four rows of X at a
// time (FP32: 256) and writes 64 bytes of a row of codes.  (4096 x 11008
// bfloat16, groups of 128 with zero points: 35.6 us, 3.2 TB/s, bound by some 20
// instructions a value; 112 us with a lane for a column's whole group.)
template <class T, class S, int GB>
__global__ void __launch_bounds__(THREADS) quantize_cols(QuantArgs p, int64_t blocks, int tiles_n, int vec) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t n0 = (b % tiles_n) * 64 + 4 * (l % 16);
    const int64_t k0 = (b / tiles_n * (THREADS / 64) + wave) * 128 + 32 * (l / 16);
    const int64_t left = p.K - k0, cols = p.N - n0;  // (0 or less: none)
    const T* x = static_cast<const T*>(p.X) + k0 * p.ldx + n0;
    T4 v[32];
    if (vec && left >= 32 && cols >= 4) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = *reinterpret_cast<const T4*>(x + i * p.ldx);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = i < left && c < cols ? x[i * p.ldx + c] : (T)0.f;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float lo = 0.f, hi = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float w = (float)v[i][c];
        lo = __builtin_fminf(lo, w);
        hi = __builtin_fmaxf(hi, w);
        sum = __builtin_fmaf(w, 0.f, sum);  // (NaN where a value is infinite or NaN)
      }
#pragma unroll
      for (int d = 16; d < GB / 2; d *= 2) {
        lo = __builtin_fminf(lo, __shfl_xor(lo, d));
        hi = __builtin_fmaxf(hi, __shfl_xor(hi, d));
        sum += __shfl_xor(sum, d);
      }
      const GroupScale<S> g(lo, hi, sum == 0.f, p.zeros != nullptr);
      if (left <= 0 || c >= cols) continue;
      uint4 w;
      unsigned* words = reinterpret_cast<unsigned*>(&w);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        words[h] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) words[h] |= g.code((float)v[8 * h + i][c]) << (4 * i);
      }
      const int64_t n = n0 + c;
      *reinterpret_cast<uint4*>(p.codes + n * p.ldq + k0 / 2) = w;
      if (k0 % GB == 0) {
        static_cast<S*>(p.scales)[n * p.lds + k0 / GB] = g.s;
        if (p.zeros) p.zeros[n * p.ldz + k0 / GB] = (uint8_t)g.zero;
      }
    }
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
    const int64_t blocks = tiles_n * (((int64_t)a.K + 2 * THREADS - 1) / (2 * THREADS));  // 128 k a wave
    const int vec = (uintptr_t)a.X % (4 * sizeof(T)) == 0 && a.ldx % 4 == 0;
    hipLaunchKernelGGL((quantize_cols<T, S, GB>), dim3((unsigned)(blocks < kMostBlocks ? blocks : kMostBlocks)), dim3(THREADS),
                       0, s, a, blocks, (int)tiles_n, vec);
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

// Values to codes and back on the conversion instructions (v_cvt_scalef32_*),
// and the loads they take: shared by the quantisation kernels and the product
// that quantises on the way.
#pragma once

#include "mx_internal.h"

namespace gemm {
namespace mx {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int DT>
constexpr int kBytes = DT == GEMM_DTYPE_F32 ? 4 : 2;

template <int FMT>
constexpr int kBlockBytes = FMT == GEMM_MX_E2M1 ? 16 : 32;

// The scale byte of a block from its largest magnitude's bit pattern (FP32;
// 255 where that is infinite or NaN).
template <int FMT>
__device__ __forceinline__ unsigned scale_byte(unsigned amax) {
  const int e = (int)(amax >> 23);
  int s;
  if constexpr (FMT == GEMM_MX_E2M1)
    s = e - 2;
  else  // 448 = 1.75 * 2^8
    s = e - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e == 255 ? 255u : (unsigned)(s < 0 ? 0 : s);
}

// FP32 bit pattern of a 16-bit magnitude.
template <int DT>
__device__ __forceinline__ unsigned widen_bits(unsigned h) {
  if constexpr (DT == GEMM_DTYPE_BF16)
    return h << 16;
  else
    return __builtin_bit_cast(unsigned, (float)__builtin_bit_cast(_Float16, (unsigned short)h));
}

// Two codes from two values: FP32 (x0, x1), or one packed 16-bit pair.  The
// result is in byte SEL (E2M1) or half-word SEL (E4M3) of the returned word,
// the rest taken from `old`.
template <int FMT, int SEL>
__device__ __forceinline__ unsigned encode2(unsigned old, float x0, float x1, float factor) {
  if constexpr (FMT == GEMM_MX_E2M1)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, x0, x1, factor, SEL);
  else
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(
                                            __builtin_bit_cast(s16x2, old), x0, x1, factor, SEL != 0));
}
template <int FMT, int DT, int SEL>
__device__ __forceinline__ unsigned encode2(unsigned old, unsigned pair, float factor) {
  if constexpr (FMT == GEMM_MX_E2M1) {
    if constexpr (DT == GEMM_DTYPE_BF16)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), factor, SEL);
    else
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, pair), factor, SEL);
  } else {
    const s16x2 o = __builtin_bit_cast(s16x2, old);
    if constexpr (DT == GEMM_DTYPE_BF16)
      return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(
                                              o, __builtin_bit_cast(bf16x2, pair), factor, SEL != 0));
    else
      return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(
                                              o, __builtin_bit_cast(f16x2, pair), factor, SEL != 0));
  }
}

__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

// Larger of each half-word.
__device__ __forceinline__ unsigned pk_umax(unsigned a, unsigned b) {
  return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// 8 consecutive values of a row as bit patterns (FP32: 8 words; 16-bit: 4).
template <int DT>
struct Eight {
  static constexpr int W = DT == GEMM_DTYPE_F32 ? 8 : 4;
  unsigned w[W];
};

// Columns c .. c+7 of a row that has n left of them (n <= 0: none, zeros).
template <int DT, bool VEC>
__device__ __forceinline__ Eight<DT> load8(const unsigned char* row, int64_t c, int64_t n) {
  Eight<DT> v;
  constexpr int B = kBytes<DT>;
  const unsigned char* p = row + c * B;
  if (VEC && n >= 8) {
#pragma unroll
    for (int i = 0; i < Eight<DT>::W / 4; ++i) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.w[4 * i + j] = x[j];
    }
    return v;
  }
#pragma unroll
  for (int i = 0; i < Eight<DT>::W; ++i) {
    if constexpr (DT == GEMM_DTYPE_F32) {
      v.w[i] = i < n ? reinterpret_cast<const unsigned*>(p)[i] : 0u;
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      const unsigned lo = 2 * i < n ? h[2 * i] : 0u, hi = 2 * i + 1 < n ? h[2 * i + 1] : 0u;
      v.w[i] = lo | (hi << 16);
    }
  }
  return v;
}

// The scale byte of a block of which the lane holds a quarter, eight values;
// its other quarters are in the lane's quad.
template <int FMT, int DT>
__device__ __forceinline__ unsigned quad_scale(const Eight<DT>& v) {
  unsigned m = 0;
  if constexpr (DT == GEMM_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, v.w[i] & 0x7fffffffu);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = pk_umax(m, v.w[i] & 0x7fff7fffu);
    m = widen_bits<DT>(umax(m & 0xffffu, m >> 16));
  }
  m = umax(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, true));  // lanes 1,0,3,2
  m = umax(m, (unsigned)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, true));  // lanes 2,3,0,1
  return scale_byte<FMT>(m);
}

// The code words of eight values in a block of scale s (E2M1: the first).
template <int FMT, int DT>
__device__ __forceinline__ u32x2 encode8(const Eight<DT>& v, unsigned s) {
  const float factor = scale_float(s);
  unsigned q[2] = {0u, 0u};
  auto put = [&](auto I, auto W, auto S) __attribute__((always_inline)) {
    constexpr int i = decltype(I)::value, w = decltype(W)::value, sel = decltype(S)::value;
    if constexpr (DT == GEMM_DTYPE_F32)
      q[w] = encode2<FMT, sel>(q[w], __builtin_bit_cast(float, v.w[2 * i]), __builtin_bit_cast(float, v.w[2 * i + 1]), factor);
    else
      q[w] = encode2<FMT, DT, sel>(q[w], v.w[i], factor);
  };
  typedef std::integral_constant<int, 0> I0;
  typedef std::integral_constant<int, 1> I1;
  typedef std::integral_constant<int, 2> I2;
  typedef std::integral_constant<int, 3> I3;
  if constexpr (FMT == GEMM_MX_E2M1) {
    put(I0{}, I0{}, I0{}); put(I1{}, I0{}, I1{}); put(I2{}, I0{}, I2{}); put(I3{}, I0{}, I3{});
  } else {
    put(I0{}, I0{}, I0{}); put(I1{}, I0{}, I1{}); put(I2{}, I1{}, I0{}); put(I3{}, I1{}, I1{});
  }
  if (s == 255u) q[0] = q[1] = 0u;
  return u32x2{q[0], q[1]};
}

}  // namespace mx
}  // namespace gemm

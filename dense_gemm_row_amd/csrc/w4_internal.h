// Internal declarations of the 4-bit weights with group scales
// (include/gemm_w4.h): kernel arguments and launch functions.
#pragma once

#include "gemm_internal.h"
#include "gemm_w4.h"

namespace gemm {
namespace w4 {

// Code bytes of a row of K values.
inline int64_t code_bytes(int64_t K) { return (K + 31) / 32 * 16; }
inline int64_t groups_of(int64_t K, int group) { return (K + group - 1) / group; }

struct QuantArgs {
  const void* X;
  int64_t ldx;
  uint8_t* codes;
  void* scales;
  uint8_t* zeros;
  int64_t ldq, lds, ldz;
  int N, K;
};

struct DequantArgs {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  int64_t ldq, lds, ldz;
  void* X;
  int64_t ldx;
  int N, K;
  // Matrices of blockIdx.y, the strides between them in bytes (codes, zeros)
  // and elements (scales, X).
  int64_t stride_q, stride_s, stride_z, stride_x;
};

struct MatmulArgs {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  int64_t ldq, lds, ldz, stride_q, stride_s, stride_z;
  const void* X;
  void* Y;
  int64_t ldx, ldy;
  int T, N, K, G;
  const int32_t* offsets;  // null: one matrix for all T rows
  int fill;
};

hipError_t launch_quantize(int dtype, int s_dtype, bool trans, int group, const QuantArgs& a, hipStream_t s);
hipError_t launch_dequantize(int dtype, int s_dtype, int group, int G, const DequantArgs& a, hipStream_t s);
// The products of few rows (w4_few.hip), activations of type DT, scales of GB k.
template <int DT, int GB>
hipError_t launch_few(const MatmulArgs& a, hipStream_t s);

}  // namespace w4
}  // namespace gemm

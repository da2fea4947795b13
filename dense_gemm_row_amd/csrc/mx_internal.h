// Internal declarations of the microscaled operators (include/gemm_mx.h):
// kernel arguments, the launch functions of mx_quant.hip, mx_matmul.hip and
// mx_wgrad.hip, and the error hook of the C-ABI layer.
#pragma once

#include "gemm_internal.h"
#include "gemm_mx.h"
#include "mx_bounds.h"

namespace gemm {

// gemm_last_error()'s message for the calling thread ("" clears it); returns
// st.  Defined in gemm_api.hip.
gemm_status_t set_last_error(gemm_status_t st, const char* msg);

namespace mx {

constexpr int BLOCK = 32;  // elements per scale

// A coded matrix: rows of whole blocks (see gemm_mx.h).
struct Coded {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ldq, lds;
};

struct QuantArgs {
  const void* X;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldx, ldq, lds;
  int rows, cols;  // of X
};

struct DequantArgs {
  Coded q;
  void* X;
  int64_t ldx;
  int rows, cols;  // of X
};

struct MatmulArgs {
  Coded a, b;
  void* C;
  int64_t ldc;
  int M, N, K;
  Epi epi;
  // A as values (launch_matmul_values): rows of ldx.
  const void* X = nullptr;
  int64_t ldx = 0;
};

struct WgradArgs {
  Coded x;
  const void* dY;
  void* dW;
  int64_t ldy, ldw;
  int T, F, N;
  float alpha, beta;
  void* workspace;  // 16-byte aligned, or null
  int64_t workspace_bytes;
};

// How a weight gradient runs on the pipelined kernel.  The workspace holds
// dY's bfloat16 terms (`planes` bytes: where dY is not bfloat16 or has rows
// of another length than whole 16 bytes), then the splits' FP32 sums.
struct WgradPlan {
  int tile = 0;     // 0: the general kernel
  int splits = 1, chunk = 0;  // tokens of a split, a multiple of 128
  int64_t planes = 0, partials = 0;
  int64_t bytes() const { return planes + partials; }
};

// The arguments of the pipelined kernel.
struct WgradPipeArgs {
  Coded x;
  const uint16_t* y;  // bfloat16 planes
  int64_t ldy, plane;
  void* C;            // dW, or the first partial sum
  int64_t ldc, c_stride;
  int T, F, N, terms, chunk;
  float alpha, beta;
};

hipError_t launch_quantize(int dtype, int format, bool trans, const QuantArgs& a, hipStream_t s);
hipError_t launch_dequantize(int dtype, int format, bool trans, const DequantArgs& a, hipStream_t s);
hipError_t launch_matmul(int c_dtype, const MatmulArgs& a, hipStream_t s);
// The same with A = X quantised on the way, for what values_fit takes.
constexpr int kValueRows = 16;
bool values_fit(int a_dtype, const MatmulArgs& a);
hipError_t launch_matmul_values(int a_dtype, int c_dtype, const MatmulArgs& a, hipStream_t s);
hipError_t launch_wgrad(int y_dtype, int c_dtype, const WgradArgs& a, hipStream_t s);
WgradPlan wgrad_plan(int y_dtype, int64_t T, int64_t F, int64_t N);
// The pipelined kernels on tiles of SIDE x SIDE (mx_matmul_pipe.hip, scales
// in pieces of SC bytes; mx_wgrad_pipe.hip), for C of type DT.
template <int DT, int SIDE, int SC>
hipError_t launch_matmul_pipe(const MatmulArgs& a, hipStream_t s);
template <int DT, int SIDE>
hipError_t launch_wgrad_pipe(const WgradPipeArgs& a, int splits, hipStream_t s);

// Output types as template arguments: GEMM_DTYPE_F32 / _F16 / _BF16.
template <int DT>
struct TypeOf;
template <>
struct TypeOf<GEMM_DTYPE_F32> { typedef float type; };
template <>
struct TypeOf<GEMM_DTYPE_F16> { typedef _Float16 type; };
template <>
struct TypeOf<GEMM_DTYPE_BF16> { typedef __bf16 type; };

// The FP32 factor of a scale byte as the conversion instructions take it:
// they read its exponent field alone (0 gives 2^-127, 255 gives NaN values;
// both checked on the device).
__device__ __forceinline__ float scale_float(unsigned byte) { return __builtin_bit_cast(float, byte << 23); }

}  // namespace mx
}  // namespace gemm

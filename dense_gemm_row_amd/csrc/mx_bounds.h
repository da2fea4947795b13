// Index arithmetic of the microscaled operators that decides which bytes are
// touched: plain integers, the same on the host, on the device and in a CPU
// test that includes this header alone.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define MX_HD __host__ __device__ inline __attribute__((always_inline))
#else
#define MX_HD inline
#endif

namespace gemm {
namespace mx {

constexpr unsigned OOB = 0x80000000u;  // offset past every descriptor's range

// Sizes go up to 2^31 - 1, so roundings up are taken in 64 bits.
MX_HD constexpr int64_t ceil_div(int64_t n, int64_t d) { return (n + d - 1) / d; }
// Blocks of 32 of a row of `cols` values.
MX_HD constexpr int64_t blocks_of(int64_t cols) { return ceil_div(cols, 32); }

// A lane's eight values of type size VB, columns c .. c+7 of row `row`, come
// in 16-byte loads (two of FP32, one of 16 bits): the byte offset of load h.
// `left` columns of the matrix are at c and beyond.  A load none of whose
// values exist is not made; of one that is made, the values past the row lie
// in the 16 aligned bytes of one that exists.
template <int VB>
MX_HD unsigned value_load(int row, int rows, unsigned row_bytes, int c, int left, int h) {
  return row < rows && left > h * (16 / VB) ? (unsigned)row * row_bytes + (unsigned)(VB * c + 16 * h) : OOB;
}

}  // namespace mx
}  // namespace gemm

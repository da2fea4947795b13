// Argument checks shared by the C-ABI entry points of the operators beside the
// plain GEMMs (mx_api.hip, grouped_api.hip, w4_api.hip).
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include "gemm_internal.h"

namespace gemm {

// gemm_last_error()'s message for the calling thread ("" clears it); returns
// st.  Defined in gemm_api.hip.
gemm_status_t set_last_error(gemm_status_t st, const char* msg);

inline gemm_status_t fail(gemm_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline gemm_status_t fail(gemm_status_t st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(st, msg);
}

inline gemm_status_t launched(hipError_t e) {
  return e == hipSuccess ? GEMM_OK : fail(GEMM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

constexpr int64_t kSizeLimit = 0x7fffffff;
inline bool size_ok(int64_t n) { return n >= 0 && n <= kSizeLimit; }
inline bool float_dtype(int d) { return d == GEMM_DTYPE_F32 || d == GEMM_DTYPE_F16 || d == GEMM_DTYPE_BF16; }
inline int64_t dtype_bytes(int d) { return d == GEMM_DTYPE_F32 ? 4 : 2; }

// A byte range [at, at + bytes): rows x row bytes at `ld` bytes.
struct Span {
  uintptr_t at;
  unsigned __int128 bytes;
};
inline Span span(const void* p, int64_t rows, int64_t row, int64_t ld) {
  if (rows <= 0 || row <= 0) return {(uintptr_t)p, 0};
  return {(uintptr_t)p, (unsigned __int128)(uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)row};
}
constexpr uint64_t kSpanLimit = (uint64_t)1 << 63;
inline bool overlap(const Span& a, const Span& b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  return a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}

// A dense rows x cols matrix of elements of es bytes.
inline gemm_status_t check_dense(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es, Span* out) {
  if (ld < (cols > 1 ? cols : 1)) return fail(GEMM_ERR_INVALID_ARG, "%s: leading dimension below its row length", name);
  if (rows > 0 && cols > 0 && !p) return fail(GEMM_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld >= (int64_t)(kSpanLimit >> 3)) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  *out = span(p, rows, cols * es, ld * es);
  if (out->bytes >= kSpanLimit) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  if (out->bytes > 0 && out->at % es != 0) return fail(GEMM_ERR_UNSUPPORTED, "%s is not aligned to its elements", name);
  return GEMM_OK;
}

}  // namespace gemm

// C-ABI entry points of the microscaled operators (include/gemm_mx.h):
// argument checks on the host, then the launch on the caller's stream.
#include <stdarg.h>
#include <stdio.h>

#include "mx_internal.h"

namespace gemm {
namespace mx {
namespace {

gemm_status_t fail(gemm_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gemm_status_t fail(gemm_status_t st, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(st, msg);
}

gemm_status_t launched(hipError_t e) {
  return e == hipSuccess ? GEMM_OK : fail(GEMM_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}

constexpr int64_t kSizeLimit = 0x7fffffff;
bool size_ok(int64_t n) { return n >= 0 && n <= kSizeLimit; }
bool float_dtype(int d) { return d == GEMM_DTYPE_F32 || d == GEMM_DTYPE_F16 || d == GEMM_DTYPE_BF16; }
int64_t dtype_bytes(int d) { return d == GEMM_DTYPE_F32 ? 4 : 2; }
int64_t row_bytes(int format, int64_t cols) { return blocks_of(cols) * (format == GEMM_MX_E2M1 ? 16 : 32); }

// A byte range [at, at + bytes): rows x row bytes at `ld` bytes.
struct Span {
  uintptr_t at;
  unsigned __int128 bytes;
};
Span span(const void* p, int64_t rows, int64_t row, int64_t ld) {
  if (rows <= 0 || row <= 0) return {(uintptr_t)p, 0};
  return {(uintptr_t)p, (unsigned __int128)(uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)row};
}
constexpr uint64_t kSpanLimit = (uint64_t)1 << 63;
bool overlap(const Span& a, const Span& b) {
  if (a.bytes == 0 || b.bytes == 0) return false;
  return a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}

// A dense rows x cols matrix of elements of es bytes.
gemm_status_t check_dense(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es, Span* out) {
  if (ld < (cols > 1 ? cols : 1)) return fail(GEMM_ERR_INVALID_ARG, "%s: leading dimension below its row length", name);
  if (rows > 0 && cols > 0 && !p) return fail(GEMM_ERR_INVALID_ARG, "%s is NULL", name);
  if (ld >= (int64_t)(kSpanLimit >> 3)) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  *out = span(p, rows, cols * es, ld * es);
  if (out->bytes >= kSpanLimit) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  if (out->bytes > 0 && out->at % es != 0) return fail(GEMM_ERR_UNSUPPORTED, "%s is not aligned to its elements", name);
  return GEMM_OK;
}

// A coded rows x cols matrix; the spans of its codes and scales.
gemm_status_t check_coded(const char* name, int format, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                          int64_t cols, int64_t ldq, int64_t lds, Span* oc, Span* os) {
  const int64_t row = row_bytes(format, cols), nb = blocks_of(cols);
  if (ldq < row) return fail(GEMM_ERR_INVALID_ARG, "%s: code rows are %lld bytes, ldq is less", name, (long long)row);
  if (lds < nb) return fail(GEMM_ERR_INVALID_ARG, "%s: scale rows are %lld bytes, lds is less", name, (long long)nb);
  if (rows > 0 && cols > 0 && (!codes || !scales)) return fail(GEMM_ERR_INVALID_ARG, "%s: codes or scales are NULL", name);
  *oc = span(codes, rows, row, ldq);
  *os = span(scales, rows, nb, lds);
  if (oc->bytes >= kSpanLimit || os->bytes >= kSpanLimit)
    return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  if (oc->bytes > 0 && ((uintptr_t)codes % 16 != 0 || ldq % 16 != 0))
    return fail(GEMM_ERR_UNSUPPORTED, "%s: codes must be 16-byte aligned with ldq a multiple of 16", name);
  return GEMM_OK;
}

gemm_status_t check_format(int dtype, int format) {
  if (!float_dtype(dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", dtype);
  if (format != GEMM_MX_E2M1 && format != GEMM_MX_E4M3) return fail(GEMM_ERR_INVALID_ARG, "unknown format %d", format);
  return GEMM_OK;
}

// Scale rows of whole 4-byte words, as the pipelined product takes them, or
// (long ones) of whole 16 bytes, as it likes them.
int64_t scale_row(int64_t cols) {
  const int64_t nb = blocks_of(cols), unit = nb < 16 ? 4 : 16;
  return (nb + unit - 1) / unit * unit;
}

// What both products share: sizes, Bt, C and the epilogue.
gemm_status_t check_product(int c_dtype, int64_t M, int64_t N, int64_t K, const uint8_t* Bt, int64_t ldbt, const uint8_t* Bs,
                            int64_t ldbs, void* C, int64_t ldc, const gemm_epilogue_t* epi, MatmulArgs* p, Span* c) {
  if (!float_dtype(c_dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", c_dtype);
  if (!size_ok(M) || !size_ok(N) || !size_ok(K)) return fail(GEMM_ERR_INVALID_ARG, "size below 0 or above 2^31-1");
  if (epi && epi->act != GEMM_ACT_NONE && epi->act != GEMM_ACT_RELU)
    return fail(GEMM_ERR_INVALID_ARG, "unknown activation %d", epi->act);
  gemm_status_t st;
  Span b, bs;
  if ((st = check_coded("Bt", GEMM_MX_E2M1, Bt, Bs, N, K, ldbt, ldbs, &b, &bs)) != GEMM_OK) return st;
  if ((st = check_dense("C", C, M, N, ldc, dtype_bytes(c_dtype), c)) != GEMM_OK) return st;
  if (overlap(*c, b) || overlap(*c, bs)) return fail(GEMM_ERR_ALIAS, "C overlaps an operand");
  *p = MatmulArgs{{}, {Bt, Bs, ldbt, ldbs}, C, ldc, (int)M, (int)N, (int)K, Epi()};
  if (epi) {
    p->epi.on = true;
    p->epi.alpha = epi->alpha;
    p->epi.beta = epi->beta;
    p->epi.bias = epi->bias;
    p->epi.act = epi->act;
    if ((uintptr_t)epi->bias % 4 != 0) return fail(GEMM_ERR_UNSUPPORTED, "bias is not aligned to its elements");
    if (overlap(*c, span(epi->bias, epi->bias ? 1 : 0, 4 * N, 4 * N))) return fail(GEMM_ERR_ALIAS, "C overlaps the bias");
  }
  return GEMM_OK;
}

}  // namespace
}  // namespace mx
}  // namespace gemm

using namespace gemm;
using namespace gemm::mx;

extern "C" {

gemm_status_t gemm_mx_quantize(int32_t dtype, int32_t format, int32_t trans, int64_t rows, int64_t cols, const void* X,
                               int64_t ldx, uint8_t* codes, int64_t ldq, uint8_t* scales, int64_t lds, void* stream) {
  set_last_error(GEMM_OK, "");
  gemm_status_t st = check_format(dtype, format);
  if (st != GEMM_OK) return st;
  if (trans != 0 && trans != 1) return fail(GEMM_ERR_INVALID_ARG, "trans is neither 0 nor 1");
  if (!size_ok(rows) || !size_ok(cols)) return fail(GEMM_ERR_INVALID_ARG, "size below 0 or above 2^31-1");
  Span x, c, s;
  if ((st = check_dense("X", X, rows, cols, ldx, dtype_bytes(dtype), &x)) != GEMM_OK) return st;
  if ((st = check_coded("output", format, codes, scales, trans ? cols : rows, trans ? rows : cols, ldq, lds, &c, &s)) != GEMM_OK)
    return st;
  if (overlap(c, x) || overlap(s, x) || overlap(c, s)) return fail(GEMM_ERR_ALIAS, "codes, scales and X overlap");
  const QuantArgs a{X, codes, scales, ldx, ldq, lds, (int)rows, (int)cols};
  return launched(launch_quantize(dtype, format, trans != 0, a, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_mx_dequantize(int32_t dtype, int32_t format, int32_t trans, int64_t rows, int64_t cols,
                                 const uint8_t* codes, int64_t ldq, const uint8_t* scales, int64_t lds, void* X,
                                 int64_t ldx, void* stream) {
  set_last_error(GEMM_OK, "");
  gemm_status_t st = check_format(dtype, format);
  if (st != GEMM_OK) return st;
  if (trans != 0 && trans != 1) return fail(GEMM_ERR_INVALID_ARG, "trans is neither 0 nor 1");
  if (!size_ok(rows) || !size_ok(cols)) return fail(GEMM_ERR_INVALID_ARG, "size below 0 or above 2^31-1");
  Span x, c, s;
  if ((st = check_dense("X", X, rows, cols, ldx, dtype_bytes(dtype), &x)) != GEMM_OK) return st;
  if ((st = check_coded("input", format, codes, scales, trans ? cols : rows, trans ? rows : cols, ldq, lds, &c, &s)) != GEMM_OK)
    return st;
  if (overlap(x, c) || overlap(x, s)) return fail(GEMM_ERR_ALIAS, "X overlaps the codes or scales");
  const DequantArgs a{{codes, scales, ldq, lds}, X, ldx, (int)rows, (int)cols};
  return launched(launch_dequantize(dtype, format, trans != 0, a, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_mx_matmul(int32_t c_dtype, int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
                             const uint8_t* As, int64_t ldas, const uint8_t* Bt, int64_t ldbt, const uint8_t* Bs,
                             int64_t ldbs, void* C, int64_t ldc, void* stream, const gemm_epilogue_t* epi) {
  set_last_error(GEMM_OK, "");
  MatmulArgs p;
  Span c, a, as;
  gemm_status_t st = check_product(c_dtype, M, N, K, Bt, ldbt, Bs, ldbs, C, ldc, epi, &p, &c);
  if (st != GEMM_OK) return st;
  if ((st = check_coded("A", GEMM_MX_E2M1, A, As, M, K, lda, ldas, &a, &as)) != GEMM_OK) return st;
  if (overlap(c, a) || overlap(c, as)) return fail(GEMM_ERR_ALIAS, "C overlaps an operand");
  p.a = Coded{A, As, lda, ldas};
  return launched(launch_matmul(c_dtype, p, static_cast<hipStream_t>(stream)));
}

int64_t gemm_mx_matmul_values_workspace_bytes(int64_t M, int64_t K) {
  if (!size_ok(M) || !size_ok(K)) return -1;
  return M * (blocks_of(K) * 16 + scale_row(K));
}

gemm_status_t gemm_mx_matmul_values(int32_t a_dtype, int32_t c_dtype, int64_t M, int64_t N, int64_t K, const void* X,
                                    int64_t ldx, const uint8_t* Bt, int64_t ldbt, const uint8_t* Bs, int64_t ldbs,
                                    void* C, int64_t ldc, void* workspace, int64_t workspace_bytes, void* stream,
                                    const gemm_epilogue_t* epi) {
  set_last_error(GEMM_OK, "");
  if (!float_dtype(a_dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", a_dtype);
  if (workspace_bytes < 0) return fail(GEMM_ERR_INVALID_ARG, "negative workspace size");
  MatmulArgs p;
  Span c, x;
  gemm_status_t st = check_product(c_dtype, M, N, K, Bt, ldbt, Bs, ldbs, C, ldc, epi, &p, &c);
  if (st != GEMM_OK) return st;
  if ((st = check_dense("X", X, M, K, ldx, dtype_bytes(a_dtype), &x)) != GEMM_OK) return st;
  if (overlap(c, x)) return fail(GEMM_ERR_ALIAS, "C overlaps X");
  if (M == 0 || N == 0) return GEMM_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  p.X = X;
  p.ldx = ldx;
  if (M <= kValueRows && values_fit(a_dtype, p)) return launched(launch_matmul_values(a_dtype, c_dtype, p, s));
  const int64_t need = gemm_mx_matmul_values_workspace_bytes(M, K);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return fail(GEMM_ERR_INVALID_ARG, "the workspace takes %lld bytes", (long long)need);
    if ((uintptr_t)workspace % 16 != 0) return fail(GEMM_ERR_INVALID_ARG, "workspace not 16-byte aligned");
    const Span k = span(workspace, 1, need, need);
    if (overlap(k, x) || overlap(k, c) || overlap(k, span(Bt, N, row_bytes(GEMM_MX_E2M1, K), ldbt)) ||
        overlap(k, span(Bs, N, blocks_of(K), ldbs)) ||
        (epi && overlap(k, span(epi->bias, epi->bias ? 1 : 0, 4 * N, 4 * N))))
      return fail(GEMM_ERR_ALIAS, "workspace overlaps an operand");
  }
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  const QuantArgs q{X, codes, codes + M * blocks_of(K) * 16, ldx, blocks_of(K) * 16, scale_row(K), (int)M, (int)K};
  p.a = Coded{q.codes, q.scales, q.ldq, q.lds};
  const hipError_t e = launch_quantize(a_dtype, GEMM_MX_E2M1, false, q, s);
  return launched(e != hipSuccess ? e : launch_matmul(c_dtype, p, s));
}

int64_t gemm_mx_wgrad_workspace_bytes(int32_t y_dtype, int64_t T, int64_t F, int64_t N) {
  if (!float_dtype(y_dtype) || !size_ok(T) || !size_ok(F) || !size_ok(N)) return -1;
  return wgrad_plan(y_dtype, T, F, N).bytes();
}

gemm_status_t gemm_mx_wgrad(int32_t y_dtype, int32_t c_dtype, int64_t T, int64_t F, int64_t N, const uint8_t* codes,
                            int64_t ldq, const uint8_t* scales, int64_t lds, const void* dY, int64_t ldy, void* dW,
                            int64_t ldw, float alpha, float beta, void* workspace, int64_t workspace_bytes,
                            void* stream) {
  set_last_error(GEMM_OK, "");
  if (!float_dtype(y_dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", y_dtype);
  if (!float_dtype(c_dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", c_dtype);
  if (!size_ok(T) || !size_ok(F) || !size_ok(N)) return fail(GEMM_ERR_INVALID_ARG, "size below 0 or above 2^31-1");
  if (workspace_bytes < 0) return fail(GEMM_ERR_INVALID_ARG, "negative workspace size");
  gemm_status_t st;
  Span c, s, y, w;
  if ((st = check_coded("checkpoint", GEMM_MX_E4M3, codes, scales, F, T, ldq, lds, &c, &s)) != GEMM_OK) return st;
  if ((st = check_dense("dY", dY, T, N, ldy, dtype_bytes(y_dtype), &y)) != GEMM_OK) return st;
  if ((st = check_dense("dW", dW, F, N, ldw, dtype_bytes(c_dtype), &w)) != GEMM_OK) return st;
  if (overlap(w, c) || overlap(w, s) || overlap(w, y)) return fail(GEMM_ERR_ALIAS, "dW overlaps an operand");
  WgradArgs p{{codes, scales, ldq, lds}, dY, dW, ldy, ldw, (int)T, (int)F, (int)N, alpha, beta, nullptr, 0};
  const int64_t need = wgrad_plan(y_dtype, T, F, N).bytes();
  if (need > 0 && workspace && workspace_bytes >= need) {
    if ((uintptr_t)workspace % 16 != 0) return fail(GEMM_ERR_INVALID_ARG, "workspace not 16-byte aligned");
    const Span k = span(workspace, 1, need, need);
    if (overlap(k, c) || overlap(k, s) || overlap(k, y) || overlap(k, w))
      return fail(GEMM_ERR_ALIAS, "workspace overlaps an operand");
    p.workspace = workspace;
    p.workspace_bytes = need;
  }
  return launched(launch_wgrad(y_dtype, c_dtype, p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// C-ABI entry points of the 4-bit weights with group scales
// (include/gemm_w4.h): argument checks on the host, then the launches on the
// caller's stream.
#include "api_checks.h"
#include "grouped_internal.h"
#include "w4_internal.h"

namespace gemm {
namespace w4 {
namespace {

constexpr int64_t kMostK = 1 << 30;

bool half_dtype(int d) { return d == GEMM_DTYPE_F16 || d == GEMM_DTYPE_BF16; }

gemm_status_t check_sizes(int64_t N, int64_t K) {
  if (!size_ok(N)) return fail(GEMM_ERR_INVALID_ARG, "N below 0 or above 2^31-1");
  if (K < 0 || K > kMostK) return fail(GEMM_ERR_INVALID_ARG, "K below 0 or above 2^30");
  return GEMM_OK;
}

// G byte ranges of `one`, `stride` bytes apart.
gemm_status_t stacked(const char* name, int64_t G, int64_t stride, int64_t es, Span* one) {
  if (one->bytes >= kSpanLimit) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  if (one->bytes == 0 || G <= 1) return GEMM_OK;
  if (stride < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative stride", name);
  one->bytes += (unsigned __int128)(uint64_t)(G - 1) * (uint64_t)stride * (unsigned)es;
  if (one->bytes >= kSpanLimit) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  return GEMM_OK;
}

struct CodedSpans {
  Span codes, scales, zeros;
  bool meets(const Span& s) const { return overlap(codes, s) || overlap(scales, s) || overlap(zeros, s); }
};

// A coded operand of G matrices of N x K.
gemm_status_t check_coded(const gemm_w4_t* q, int64_t G, int64_t N, int64_t K, CodedSpans* o) {
  if (!q) return fail(GEMM_ERR_INVALID_ARG, "the weights' description is NULL");
  if (q->group != 32 && q->group != 64 && q->group != 128)
    return fail(GEMM_ERR_INVALID_ARG, "groups of %d: 32, 64 or 128", q->group);
  const int64_t row = code_bytes(K), ng = groups_of(K, q->group);
  if (q->ldq < row) return fail(GEMM_ERR_INVALID_ARG, "code rows are %lld bytes, ldq is less", (long long)row);
  if (q->lds < ng) return fail(GEMM_ERR_INVALID_ARG, "scale rows are %lld long, lds is less", (long long)ng);
  if (q->zeros && q->ldz < ng) return fail(GEMM_ERR_INVALID_ARG, "zero point rows are %lld long, ldz is less", (long long)ng);
  if (q->lds >= (int64_t)(kSpanLimit >> 3)) return fail(GEMM_ERR_INVALID_ARG, "scales: byte range reaches 2^63");
  const int64_t rows = G > 0 ? N : 0;
  if (rows > 0 && K > 0 && (!q->codes || !q->scales)) return fail(GEMM_ERR_INVALID_ARG, "codes or scales are NULL");
  o->codes = span(q->codes, rows, row, q->ldq);
  o->scales = span(q->scales, rows, 2 * ng, 2 * q->lds);
  o->zeros = span(q->zeros, q->zeros ? rows : 0, ng, q->ldz);
  gemm_status_t st;
  if ((st = stacked("codes", G, q->stride_q, 1, &o->codes)) != GEMM_OK) return st;
  if ((st = stacked("scales", G, q->stride_s, 2, &o->scales)) != GEMM_OK) return st;
  if ((st = stacked("zeros", G, q->stride_z, 1, &o->zeros)) != GEMM_OK) return st;
  if (o->codes.bytes > 0 && ((uintptr_t)q->codes % 16 != 0 || q->ldq % 16 != 0 || (G > 1 && q->stride_q % 16 != 0)))
    return fail(GEMM_ERR_UNSUPPORTED, "codes must be 16-byte aligned with ldq and stride multiples of 16");
  if (o->scales.bytes > 0 && (uintptr_t)q->scales % 2 != 0)
    return fail(GEMM_ERR_UNSUPPORTED, "scales are not aligned to their elements");
  return GEMM_OK;
}

// The workspace of the products with many rows: G dequantised matrices, rows
// of whole 16 bytes.
int64_t row_values(int64_t K) { return (K + 7) / 8 * 8; }
int64_t workspace_for(bool many, int64_t G, int64_t N, int64_t K) {
  const unsigned __int128 n = many ? (unsigned __int128)(uint64_t)G * (uint64_t)N * (uint64_t)(2 * row_values(K)) : 0;
  return n < kSpanLimit ? (int64_t)n : -1;
}
gemm_status_t check_workspace(const void* p, int64_t bytes, int64_t need, const CodedSpans& q, const Span& x, const Span& y,
                              const Span& offsets) {
  if (need < 0) return fail(GEMM_ERR_INVALID_ARG, "the dequantised weights' bytes reach 2^63");
  if (need == 0) return GEMM_OK;
  if (!p || bytes < need) return fail(GEMM_ERR_INVALID_ARG, "the workspace takes %lld bytes", (long long)need);
  if ((uintptr_t)p % 16 != 0) return fail(GEMM_ERR_INVALID_ARG, "workspace not 16-byte aligned");
  const Span k = span(p, 1, need, need);
  if (overlap(k, x) || overlap(k, y) || overlap(k, offsets) || q.meets(k)) return fail(GEMM_ERR_ALIAS, "workspace overlaps an operand");
  return GEMM_OK;
}

bool many_rows(int64_t T, int64_t G, int64_t K) { return G > 0 && K > 0 && T > GEMM_W4_ROWS * G; }

MatmulArgs args_of(const gemm_w4_t* q, const void* X, int64_t ldx, void* Y, int64_t ldy, int64_t T, int64_t N, int64_t K,
                   int64_t G, const int32_t* offsets, int fill) {
  return {q->codes, q->scales, q->zeros, q->ldq, q->lds, q->ldz, q->stride_q, q->stride_s, q->stride_z,
          X, Y, ldx, ldy, (int)T, (int)N, (int)K, (int)G, offsets, fill};
}

template <int DT>
hipError_t by_group(int group, const MatmulArgs& a, hipStream_t s) {
  if (group == 32) return launch_few<DT, 32>(a, s);
  return group == 64 ? launch_few<DT, 64>(a, s) : launch_few<DT, 128>(a, s);
}
hipError_t few_rows(int dtype, int group, const MatmulArgs& a, hipStream_t s) {
  return dtype == GEMM_DTYPE_BF16 ? by_group<GEMM_DTYPE_BF16>(group, a, s) : by_group<GEMM_DTYPE_F16>(group, a, s);
}

// All weights for the products with many rows, rounded to the activations'
// type: s (q - z) has up to 12 significant bits (binary16: 15), the type 8 (11).
// A product of 4096 k is then off by 0.0022 (0.00028) of its size, from the codes
// by 0.00166 (0.00021), the rounding of the result itself.  The price of a library's
// product at its full rate: 512 rows, 4096 x 11008, 75.9 us, from the codes, read
// once more for each 128 rows, 160.7; 1024 rows 106 and 320; 256 rows 63.6 and 80.6
// (but of 4096 x 4096 53.5 and 39.7).
hipError_t dequantize_all(int dtype, const gemm_w4_t* q, int64_t G, int64_t N, int64_t K, void* out, hipStream_t s) {
  const int64_t ld = row_values(K);
  const DequantArgs d{q->codes, q->scales, q->zeros, q->ldq, q->lds, q->ldz, out, ld, (int)N, (int)K,
                      q->stride_q, q->stride_s, q->stride_z, N * ld};
  return launch_dequantize(dtype, dtype, q->group, (int)G, d, s);
}

}  // namespace
}  // namespace w4
}  // namespace gemm

using namespace gemm;
using namespace gemm::w4;

extern "C" {

gemm_status_t gemm_w4_quantize(int32_t dtype, int32_t s_dtype, int32_t trans, int64_t N, int64_t K, const void* X, int64_t ldx,
                               const gemm_w4_t* q, void* stream) {
  set_last_error(GEMM_OK, "");
  if (!float_dtype(dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", dtype);
  if (!half_dtype(s_dtype)) return fail(GEMM_ERR_INVALID_ARG, "the scales' type %d is not F16 or BF16", s_dtype);
  if (trans != 0 && trans != 1) return fail(GEMM_ERR_INVALID_ARG, "trans is neither 0 nor 1");
  gemm_status_t st;
  CodedSpans c;
  Span x;
  if ((st = w4::check_sizes(N, K)) != GEMM_OK) return st;
  if ((st = check_dense("X", X, trans ? K : N, trans ? N : K, ldx, dtype_bytes(dtype), &x)) != GEMM_OK) return st;
  if ((st = w4::check_coded(q, 1, N, K, &c)) != GEMM_OK) return st;
  if (c.meets(x) || overlap(c.codes, c.scales) || overlap(c.codes, c.zeros) || overlap(c.scales, c.zeros))
    return fail(GEMM_ERR_ALIAS, "codes, scales, zeros and X overlap");
  const QuantArgs a{X, ldx, const_cast<uint8_t*>(q->codes), const_cast<void*>(q->scales), const_cast<uint8_t*>(q->zeros),
                    q->ldq, q->lds, q->ldz, (int)N, (int)K};
  return launched(launch_quantize(dtype, s_dtype, trans != 0, q->group, a, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_w4_dequantize(int32_t dtype, int32_t s_dtype, int64_t N, int64_t K, const gemm_w4_t* q, void* X, int64_t ldx,
                                 void* stream) {
  set_last_error(GEMM_OK, "");
  if (!float_dtype(dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", dtype);
  if (!half_dtype(s_dtype)) return fail(GEMM_ERR_INVALID_ARG, "the scales' type %d is not F16 or BF16", s_dtype);
  gemm_status_t st;
  CodedSpans c;
  Span x;
  if ((st = w4::check_sizes(N, K)) != GEMM_OK) return st;
  if ((st = w4::check_coded(q, 1, N, K, &c)) != GEMM_OK) return st;
  if ((st = check_dense("X", X, N, K, ldx, dtype_bytes(dtype), &x)) != GEMM_OK) return st;
  if (c.meets(x)) return fail(GEMM_ERR_ALIAS, "X overlaps the codes, scales or zeros");
  const DequantArgs a{q->codes, q->scales, q->zeros, q->ldq, q->lds, q->ldz, X, ldx, (int)N, (int)K, 0, 0, 0, 0};
  return launched(launch_dequantize(dtype, s_dtype, q->group, 1, a, static_cast<hipStream_t>(stream)));
}

int64_t gemm_w4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!size_ok(M) || !size_ok(N) || K < 0 || K > kMostK) return -1;
  return workspace_for(many_rows(M, 1, K), 1, N, K);
}

gemm_status_t gemm_w4_matmul(int32_t dtype, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const gemm_w4_t* q,
                             void* Y, int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream) {
  set_last_error(GEMM_OK, "");
  if (!half_dtype(dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F16 or BF16", dtype);
  if (!size_ok(M)) return fail(GEMM_ERR_INVALID_ARG, "M below 0 or above 2^31-1");
  if (workspace_bytes < 0) return fail(GEMM_ERR_INVALID_ARG, "negative workspace size");
  gemm_status_t st;
  CodedSpans c;
  Span x, y;
  if ((st = w4::check_sizes(N, K)) != GEMM_OK) return st;
  if ((st = check_dense("X", X, M, K, ldx, 2, &x)) != GEMM_OK) return st;
  if ((st = w4::check_coded(q, 1, N, K, &c)) != GEMM_OK) return st;
  if ((st = check_dense("Y", Y, M, N, ldy, 2, &y)) != GEMM_OK) return st;
  if (overlap(y, x) || c.meets(y)) return fail(GEMM_ERR_ALIAS, "Y overlaps an operand");
  if (M == 0 || N == 0) return GEMM_OK;
  const int64_t need = gemm_w4_matmul_workspace_bytes(M, N, K);
  if ((st = check_workspace(workspace, workspace_bytes, need, c, x, y, Span{0, 0})) != GEMM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!many_rows(M, 1, K))
    return launched(few_rows(dtype, q->group, args_of(q, X, ldx, Y, ldy, M, N, K, 1, nullptr, 0), s));
  if ((st = launched(dequantize_all(dtype, q, 1, N, K, workspace, s))) != GEMM_OK) return st;
  // (Rows of X or Y that do not begin on 16 bytes: 300 rows, 8192 x 4095, 704 us on
  // the plain product, 81 on the grouped one of a single group; 320 rows, 149 x
  // 1952, 171 and 18.)
  if ((uintptr_t)X % 16 != 0 || ldx % 8 != 0 || K % 8 != 0 || (uintptr_t)Y % 16 != 0 || ldy % 8 != 0 || N % 8 != 0)
    return launched(grouped::launch_matmul(
        dtype, dtype, grouped::MatmulArgs{nullptr, X, workspace, Y, ldx, row_values(K), 0, ldy, 1,
                                          (int)M, (int)N, (int)K, 0, 1}, s));
  return (dtype == GEMM_DTYPE_BF16 ? gemm_bf16_bt : gemm_f16_bt)(M, N, K, static_cast<const uint16_t*>(X), ldx,
                                                                 static_cast<const uint16_t*>(workspace), row_values(K),
                                                                 static_cast<uint16_t*>(Y), ldy, stream, nullptr);
}

int64_t gemm_w4_grouped_workspace_bytes(int64_t G, int64_t T, int64_t N, int64_t K) {
  if (G < 0 || G > grouped::kMostGroups || !size_ok(T) || !size_ok(N) || K < 0 || K > kMostK) return -1;
  return workspace_for(many_rows(T, G, K), G, N, K);
}

gemm_status_t gemm_w4_grouped(int32_t dtype, int64_t G, int64_t T, int64_t N, int64_t K, const int32_t* offsets, const void* X,
                              int64_t ldx, const gemm_w4_t* q, void* Y, int64_t ldy, int32_t fill, void* workspace,
                              int64_t workspace_bytes, void* stream) {
  set_last_error(GEMM_OK, "");
  if (!half_dtype(dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F16 or BF16", dtype);
  if (G < 0 || G > grouped::kMostGroups)
    return fail(GEMM_ERR_INVALID_ARG, "%lld groups: 0 to %lld", (long long)G, (long long)grouped::kMostGroups);
  if (!size_ok(T)) return fail(GEMM_ERR_INVALID_ARG, "T below 0 or above 2^31-1");
  if (fill != 0 && fill != 1) return fail(GEMM_ERR_INVALID_ARG, "fill is neither 0 nor 1");
  if (workspace_bytes < 0) return fail(GEMM_ERR_INVALID_ARG, "negative workspace size");
  if (!offsets) return fail(GEMM_ERR_INVALID_ARG, "offsets is NULL");
  if ((uintptr_t)offsets % 4 != 0) return fail(GEMM_ERR_UNSUPPORTED, "offsets is not aligned to its elements");
  gemm_status_t st;
  CodedSpans c;
  Span x, y;
  const Span o = span(offsets, 1, 4 * (G + 1), 4 * (G + 1));
  if ((st = w4::check_sizes(N, K)) != GEMM_OK) return st;
  if ((st = check_dense("X", X, T, K, ldx, 2, &x)) != GEMM_OK) return st;
  if ((st = w4::check_coded(q, G, N, K, &c)) != GEMM_OK) return st;
  if ((st = check_dense("Y", Y, T, N, ldy, 2, &y)) != GEMM_OK) return st;
  if (overlap(y, x) || c.meets(y) || overlap(y, o)) return fail(GEMM_ERR_ALIAS, "Y overlaps an operand");
  if (T == 0 || N == 0) return GEMM_OK;
  const int64_t need = gemm_w4_grouped_workspace_bytes(G, T, N, K);
  if ((st = check_workspace(workspace, workspace_bytes, need, c, x, y, o)) != GEMM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!many_rows(T, G, K))
    return launched(few_rows(dtype, q->group, args_of(q, X, ldx, Y, ldy, T, N, K, G, offsets, fill), s));
  if ((st = launched(dequantize_all(dtype, q, G, N, K, workspace, s))) != GEMM_OK) return st;
  return gemm_grouped_matmul(dtype, dtype, 1, G, T, N, K, offsets, X, ldx, workspace, row_values(K), N * row_values(K), Y, ldy,
                             fill, stream);
}

}  // extern "C"

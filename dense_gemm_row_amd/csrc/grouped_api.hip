// C-ABI entry points of the grouped products (include/gemm_grouped.h):
// argument checks on the host, then the launch on the caller's stream.
#include "api_checks.h"
#include "grouped_internal.h"

namespace gemm {
namespace grouped {
namespace {

gemm_status_t check_types(int dtype, int c_dtype) {
  if (!float_dtype(dtype)) return fail(GEMM_ERR_INVALID_ARG, "type %d is not F32, F16 or BF16", dtype);
  if (c_dtype != dtype && c_dtype != GEMM_DTYPE_F32)
    return fail(GEMM_ERR_INVALID_ARG, "the result's type %d is neither the operands' nor F32", c_dtype);
  return GEMM_OK;
}

gemm_status_t check_sizes(int64_t G, int64_t T, int64_t K, int64_t N, const int32_t* offsets, Span* o) {
  if (G < 0 || G > kMostGroups) return fail(GEMM_ERR_INVALID_ARG, "%lld groups: 0 to %lld", (long long)G, (long long)kMostGroups);
  if (!size_ok(T) || !size_ok(K) || !size_ok(N)) return fail(GEMM_ERR_INVALID_ARG, "size below 0 or above 2^31-1");
  if (!offsets) return fail(GEMM_ERR_INVALID_ARG, "offsets is NULL");
  if ((uintptr_t)offsets % 4 != 0) return fail(GEMM_ERR_UNSUPPORTED, "offsets is not aligned to its elements");
  *o = span(offsets, 1, 4 * (G + 1), 4 * (G + 1));
  return GEMM_OK;
}

// G matrices of rows x cols, `stride` elements apart; `apart`: they must lie one
// behind another (an output's).
gemm_status_t check_stack(const char* name, const void* p, int64_t G, int64_t rows, int64_t cols, int64_t ld, int64_t stride,
                          int64_t es, bool apart, Span* out) {
  Span one;
  if (stride < 0) return fail(GEMM_ERR_INVALID_ARG, "%s: negative stride", name);
  const gemm_status_t st = check_dense(name, p, G > 0 ? rows : 0, cols, ld, es, &one);
  if (st != GEMM_OK) return st;
  *out = one;
  if (one.bytes == 0 || G <= 1) return GEMM_OK;
  if (stride >= (int64_t)(kSpanLimit >> 3)) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  if (apart && (unsigned __int128)(uint64_t)stride * (unsigned)es < one.bytes)
    return fail(GEMM_ERR_INVALID_ARG, "%s: the matrices of two groups overlap, or lie between one another's rows", name);
  out->bytes += (unsigned __int128)(uint64_t)(G - 1) * (uint64_t)(stride * es);
  if (out->bytes >= kSpanLimit) return fail(GEMM_ERR_INVALID_ARG, "%s: byte range reaches 2^63", name);
  return GEMM_OK;
}

// What the pipelined kernels take: 16-bit operands in whole 16-byte pieces,
// a tile's and a slice's rows within 31 bits of bytes, and a grid within the
// runtime's bounds.
constexpr int64_t kFar = 1 << 20;
constexpr int64_t kMostTiles = (1ll << 32) / 256 - 256;
bool pieces(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0 && ld < kFar; }

bool pipe_fits(int dtype, const MatmulArgs& a, int side) {
  const int64_t tiles_n = ((int64_t)a.N + 127) / 128, tiles_m = most_tiles(a.T, a.G, a.fill, side);
  return dtype != GEMM_DTYPE_F32 && a.K % 8 == 0 && (a.trans_w || a.N % 8 == 0) && pieces(a.X, a.ldx) && pieces(a.W, a.ldw) &&
         (a.G <= 1 || a.stride_w % 8 == 0) && a.ldy < kFar && (tiles_m == 0 || tiles_n <= kMostTiles / tiles_m);
}
bool pipe_fits(int dtype, const WgradArgs& a) {
  const int64_t tiles = (((int64_t)a.K + 127) / 128) * (((int64_t)a.N + 127) / 128);
  return dtype != GEMM_DTYPE_F32 && a.K % 8 == 0 && a.N % 8 == 0 && pieces(a.X, a.ldx) && pieces(a.dY, a.ldy) && a.ldw < kFar &&
         a.T < (1 << 30) && (a.G == 0 || tiles <= kMostTiles / a.G);
}

template <int DT, int CT>
hipError_t on_tile(int side, const MatmulArgs& a, hipStream_t s) {
  return side == 128 ? launch_pipe<DT, CT, 128>(a, s) : launch_pipe<DT, CT, 256>(a, s);
}
template <int DT, int CT>
hipError_t on_tile(int side, const WgradArgs& a, hipStream_t s) {
  return side == 128 ? launch_pipe<DT, CT, 128>(a, s) : launch_pipe<DT, CT, 256>(a, s);
}
template <class Args>
hipError_t pipelined(int dtype, int c_dtype, int side, const Args& a, hipStream_t s) {
  if (dtype == GEMM_DTYPE_BF16)
    return c_dtype == GEMM_DTYPE_F32 ? on_tile<GEMM_DTYPE_BF16, GEMM_DTYPE_F32>(side, a, s)
                                     : on_tile<GEMM_DTYPE_BF16, GEMM_DTYPE_BF16>(side, a, s);
  return c_dtype == GEMM_DTYPE_F32 ? on_tile<GEMM_DTYPE_F16, GEMM_DTYPE_F32>(side, a, s)
                                   : on_tile<GEMM_DTYPE_F16, GEMM_DTYPE_F16>(side, a, s);
}

// Time of `tiles` tiles, `at_once` of them at a time, half a round lost at the
// end; `fixed` us a tile beside `per_slice` for each of its slices of 64 k.
double tile_us(double tiles, int at_once, double fixed, double per_slice, double slices) {
  const double rounds = tiles / at_once + 0.5;
  return (rounds < 1. ? 1. : rounds) * (fixed + per_slice * slices);
}

// The tile of least time by a model of the measurements: 256 x 256, one
// workgroup a CU, 1.35 us a slice and 13 beside; 128 x 128, two a CU, 1.1 us (0.66
// one a CU) and 5.5, or with four stages (`alone`) 0.34 and 4.8; 16 x 64 (16),
// one a CU, 0.2 us a slice and 3; none faster than 5.2 TB/s of the weights that
// it reads, 16 x 64 those of each of its row tiles.  (64 groups of 256 rows, K
// 1024, N 2048: 128 x 128 130 us, 256 x 256 140; 8 groups of 256, 4096 x 4096: 139
// and 103; 32 groups of 128, 2048 x 1024: 47 and 60.  16 x 64 and 128 x 128: 32
// groups of one row, 2048 x 1024, 18.6 and 31.6 us; 16 of 31, 1000 x 1000, 20.4 and
// 12.0; 8 of 12, 4096 x 1024, 15.3 and 25.3; 64 of 16, 1024 x 2048, 85 and 64.)
int tile_for(const MatmulArgs& a) {
  const double slices = tiles_along(a.K, 64), groups = a.T < a.G ? a.T : a.G, of_one = 2. * a.N * a.K / 5.2e6, read = groups * of_one;
  auto us = [&](int side, int at_once, double fixed, double per_slice, double lone) {
    const double tiles = likely_tiles(a, side);
    return tile_us(tiles, at_once, fixed, tiles <= kCus ? lone : per_slice, slices);
  };
  const double m = a.T / 16. + 0.5 * groups, read16 = (m < a.T ? m : a.T) * of_one;
  const double us16 = tile_us(m * tiles_along(a.N, 64), 256, 3., 0.2, slices);
  const double us128 = alone(a) ? 4.8 + 0.34 * slices : us(128, 512, 5.5, 1.1, 0.66), us256 = us(256, 256, 13., 1.35, 1.35);
  if ((us16 > read16 ? us16 : read16) < (us128 > read ? us128 : read) && us16 < us256) return 16;
  return us256 < us128 ? 256 : 128;
}
// The gradient's likewise: a tile writes as many results however few rows its
// group has, 14 us beside 1.35 a slice on 256 x 256, 6.4 beside 0.82 on 128 x 128;
// groups that differ in rows lose three quarters of a round.  (8 groups of 2048
// rows on average, 4096 x 4096, FP32: 460 us on 256 and 540 on 128; 2048 x 2048: 158
// and 132; of 512, 2048 x 2048: 50 and 51; 64 of 256, 1024 x 1024: 88 and 80.)
int tile_for(const WgradArgs& a) {
  const double slices = (double)a.T / (a.G > 0 ? a.G : 1) / 64;
  auto us = [&](int side, int at_once, double fixed, double per_slice) {
    const double rounds = likely_tiles(a, side) / at_once;
    return (a.G > 1 ? rounds + 0.75 : __builtin_ceil(rounds)) * (fixed + per_slice * (slices < 2 ? 2 : slices));
  };
  return us(256, 256, 14., 1.35) < us(128, 512, 6.4, 0.82) ? 256 : 128;
}

hipError_t launch(int dtype, int c_dtype, const WgradArgs& a, hipStream_t s) {
  return pipe_fits(dtype, a) ? pipelined(dtype, c_dtype, tile_for(a), a, s) : launch_general(dtype, c_dtype, a, s);
}

}  // namespace

hipError_t launch_matmul(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s) {
  const int side = tile_for(a);
  if (!pipe_fits(dtype, a, side)) return launch_general(dtype, c_dtype, a, s);
  return side == 16 ? launch_few(dtype, c_dtype, a, s) : pipelined(dtype, c_dtype, side, a, s);
}

}  // namespace grouped
}  // namespace gemm

using namespace gemm;
using namespace gemm::grouped;

extern "C" {

gemm_status_t gemm_grouped_matmul(int32_t dtype, int32_t c_dtype, int32_t trans_w, int64_t G, int64_t T, int64_t N, int64_t K,
                                  const int32_t* offsets, const void* X, int64_t ldx, const void* W, int64_t ldw,
                                  int64_t stride_w, void* Y, int64_t ldy, int32_t fill, void* stream) {
  set_last_error(GEMM_OK, "");
  gemm_status_t st = check_types(dtype, c_dtype);
  if (st != GEMM_OK) return st;
  if (trans_w != 0 && trans_w != 1) return fail(GEMM_ERR_INVALID_ARG, "trans_w is neither 0 nor 1");
  if (fill != 0 && fill != 1) return fail(GEMM_ERR_INVALID_ARG, "fill is neither 0 nor 1");
  Span o, x, w, y;
  if ((st = check_sizes(G, T, K, N, offsets, &o)) != GEMM_OK) return st;
  const int64_t es = dtype_bytes(dtype);
  if ((st = check_dense("X", X, T, K, ldx, es, &x)) != GEMM_OK) return st;
  if ((st = check_stack("W", W, G, trans_w ? N : K, trans_w ? K : N, ldw, stride_w, es, false, &w)) != GEMM_OK) return st;
  if ((st = check_dense("Y", Y, T, N, ldy, dtype_bytes(c_dtype), &y)) != GEMM_OK) return st;
  if (overlap(y, x) || overlap(y, w) || overlap(y, o)) return fail(GEMM_ERR_ALIAS, "Y overlaps an operand");
  const MatmulArgs a{offsets, X, W, Y, ldx, ldw, stride_w, ldy, (int)G, (int)T, (int)N, (int)K, fill, trans_w};
  return launched(grouped::launch_matmul(dtype, c_dtype, a, static_cast<hipStream_t>(stream)));
}

gemm_status_t gemm_grouped_wgrad(int32_t dtype, int32_t c_dtype, int64_t G, int64_t T, int64_t K, int64_t N,
                                 const int32_t* offsets, const void* X, int64_t ldx, const void* dY, int64_t ldy, void* dW,
                                 int64_t ldw, int64_t stride_w, float alpha, float beta, void* stream) {
  set_last_error(GEMM_OK, "");
  gemm_status_t st = check_types(dtype, c_dtype);
  if (st != GEMM_OK) return st;
  Span o, x, y, w;
  if ((st = check_sizes(G, T, K, N, offsets, &o)) != GEMM_OK) return st;
  const int64_t es = dtype_bytes(dtype);
  if ((st = check_dense("X", X, T, K, ldx, es, &x)) != GEMM_OK) return st;
  if ((st = check_dense("dY", dY, T, N, ldy, es, &y)) != GEMM_OK) return st;
  if ((st = check_stack("dW", dW, G, K, N, ldw, stride_w, dtype_bytes(c_dtype), true, &w)) != GEMM_OK) return st;
  if (overlap(w, x) || overlap(w, y) || overlap(w, o)) return fail(GEMM_ERR_ALIAS, "dW overlaps an operand");
  const WgradArgs a{offsets, X, dY, dW, ldx, ldy, ldw, stride_w, (int)G, (int)T, (int)K, (int)N, alpha, beta};
  return launched(grouped::launch(dtype, c_dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

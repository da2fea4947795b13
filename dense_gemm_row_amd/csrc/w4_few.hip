// Products of few rows with 4-bit weights (include/gemm_w4.h), dense and
// grouped: Y[t] = X[t] x W^T with
//   W[n][k] = s[n][j] (q[n][k] - z[n][j]),  j = k / group, so that
//   Y[t][n] = sum_j s[n][j] (sum_{k in j} q X[t][k] - z[n][j] sum_{k in j} X[t][k]).
//  * A workgroup of 8 or 16 waves computes 16 MB rows x 16 NB NW columns: KW waves
//    along k, whose sums are added in order through LDS at the end, times NW
//    along the columns.  A wave's codes are read straight into registers, 16
//    rows of SPAN / 2 bytes; the waves of one part of k share X through LDS.
//  * A lane loads 16 bytes of codes, lane group q (of four) the q-th 32 k of 128,
//    a word of 8 codes for each matrix instruction; any order of k common to
//    both operands will do.  For groups shorter than 128 the lane groups
//    exchange words, four instructions for four words, so that each matrix
//    instruction has 32 k of one group.  (Loads of group / 8 bytes kept the cache
//    busy with 16 rows each: 64 experts of 2048 x 2048, 512 rows, groups of 32, 111
//    us.)
//  * A code q goes to the top of a significand as 16 + q, exact in both types:
//    four shifts and four mask-and-or for 8 codes.  (The conversions from E4M3,
//    which reads a byte 0 .. 15 as that number times 2^-9, took a mask, two
//    permutes and four conversions for the same time.)  Of the sum, 16 + z times
//    the sum of X is taken off, which one more matrix instruction a step gives,
//    with ones for weights, in the layout of the other sums; zero point and
//    scale are two fused operations a value.  A result that is not finite then is
//    taken from the definition instead (`defined`).
// Bound by the latency of its loads where there are few tiles (4096 x 4096, one
// row: 7.2 us, 1.2 TB/s), by instructions and waits for loads where there are
// many (64 experts of 2048 x 2048, groups of 128: a row each 42 us, 3.4 TB/s; 512 rows
// as a router deals them 49, groups of 32 58 to 60).
// One file for every combination of W4_TYPE (type of the activations) and
// W4_GROUP (k of a scale): compiled once for each.
#if !defined(W4_TYPE) || !defined(W4_GROUP)
#error "compiled once for every W4_TYPE and W4_GROUP"
#endif

#include <utility>

#include "grouped_internal.h"
#include "w4_internal.h"

namespace gemm {
namespace w4 {
namespace {

constexpr unsigned OOB = 0x80000000u;  // offset past every descriptor's range
constexpr int64_t kMostItems = 1ll << 31;  // work-items of a grid (the runtime takes fewer than 2^32); workgroups walk on from there
constexpr int64_t kFar = 1 << 22;  // leading dimensions below it: a tile's rows and columns are within 31 bits of bytes

template <class F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each(f, std::make_integer_sequence<int, N>{});
}

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Eight codes q as the eight numbers 16 + q of the type, codes 0, 4, 1, 5, 2, 6,
// 3, 7 in order: a code goes to the four highest bits of the significand of
// 16 = 2^4 (bfloat16 0x4180, binary16 0x4c00).
template <bool BF>
__device__ __forceinline__ u32x4 widen(unsigned w) {
  if constexpr (BF)
    return u32x4{(w << 3 & 0x00780078u) | 0x41804180u, (w >> 1 & 0x00780078u) | 0x41804180u,
                 (w >> 5 & 0x00780078u) | 0x41804180u, (w >> 9 & 0x00780078u) | 0x41804180u};
  else
    return u32x4{(w << 6 & 0x03c003c0u) | 0x4c004c00u, (w << 2 & 0x03c003c0u) | 0x4c004c00u,
                 (w >> 2 & 0x03c003c0u) | 0x4c004c00u, (w >> 6 & 0x03c003c0u) | 0x4c004c00u};
}

// Word i of lane group q (16 lanes) becomes word q of lane group i.
__device__ __forceinline__ void exchange(unsigned (&w)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto swap32 = [](unsigned& a, unsigned& b) __attribute__((always_inline)) {
    const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
    a = t[0], b = t[1];
  };
  auto swap16 = [](unsigned& a, unsigned& b) __attribute__((always_inline)) {
    const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a, b, false, false));
    a = t[0], b = t[1];
  };
  swap32(w[0], w[2]);
  swap32(w[1], w[3]);
  swap16(w[0], w[1]);
  swap16(w[2], w[3]);
#endif
}

// Eight values in the same order.
__device__ __forceinline__ u32x4 reorder(u32x4 x) {
#if defined(__HIP_DEVICE_COMPILE__)
  return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
#else
  return x;
#endif
}

// WAVES waves are KW along k times NW along the columns, each with NB blocks of
// 16 columns; SPAN k at a time.
template <int GB_, int MB_, int NB_, int KW_, int WAVES_ = 8>
struct Shape {
  static constexpr int GB = GB_, MB = MB_, NB = NB_, KW = KW_, WAVES = WAVES_, NW = WAVES / KW_;
  static constexpr int SPAN = MB == 1 ? 256 : 128;
  static constexpr int V = GB / 32;         // matrix instructions of a group
  static constexpr int GROUPS = SPAN / GB;  // groups of a span
  static constexpr int ROWS = 16 * MB, COLS = 16 * NB * NW;
  static constexpr bool SHARED = NW > 1;    // X goes through LDS
  static constexpr int X_BYTES = ROWS * SPAN * 2, XL = X_BYTES / 1024 / NW;  // of a span; a wave's loads of it
  static constexpr int X_LDS = SHARED ? 2 * KW * X_BYTES : 0, SUMS = 4 * KW * ROWS * COLS;
  static constexpr int LDS = X_LDS > SUMS ? X_LDS : SUMS;
  static_assert(GROUPS >= 1 && XL >= 1 && XL * NW * 1024 == X_BYTES && LDS <= 160 * 1024, "shape");
  // The 8 k (from the span's first on, over 8) of lane group q in the matrix
  // instruction `step`: a lane's 16 bytes of codes are 32 k in a row, one such
  // run after another in the steps of a group of 128; of shorter groups, the
  // four lane groups have exchanged their words, so that a step is 32 k.
  __host__ __device__ static constexpr int chunk(int step, int q) {
    return GB == 128 ? 16 * (step / 4) + 4 * q + step % 4 : 4 * step + q;
  }
  // 16-byte chunk c of row m of a span of X in LDS: 16 rows' reads of one
  // chunk fall on distinct banks.
  __device__ static constexpr int x_byte(int m, int c) { return 2 * SPAN * m + 16 * (c ^ (m % 16)); }
};

// What a lane reads of one span: its columns' words of codes, their scales and
// zero points as they lie in memory, and pieces of X (not SHARED: its operands,
// [group][instruction][block]).
template <class S>
struct Codes {
  unsigned w[S::NB][S::SPAN / 128][4], s[S::NB][(S::GROUPS + 1) / 2], z[S::NB][(S::GROUPS + 3) / 4];
  u32x4 x[S::XL];
};

// How a lane reads: ANY by element (X in pieces where it can); SPANS, in 16-byte
// pieces wherever they begin; WHOLE, aligned pieces through descriptors whose range ends them.
enum Reads { ANY, SPANS, WHOLE };

// N words (of BYTES bytes, 1 to 4 N) at an offset of a buffer.
template <int N, int BYTES = 4 * N>
__device__ __forceinline__ void buffer_words(__amdgpu_buffer_rsrc_t from, unsigned off, unsigned (&to)[N]) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (BYTES == 1) to[0] = __builtin_amdgcn_raw_buffer_load_b8(from, off, 0, 0);
  else if constexpr (BYTES == 2) to[0] = __builtin_amdgcn_raw_buffer_load_b16(from, off, 0, 0);
  else if constexpr (BYTES == 4) to[0] = __builtin_amdgcn_raw_buffer_load_b32(from, off, 0, 0);
  else if constexpr (BYTES == 8) __builtin_memcpy(to, &(const u32x2&)__builtin_amdgcn_raw_buffer_load_b64(from, off, 0, 0), 8);
  else __builtin_memcpy(to, &(const u32x4&)__builtin_amdgcn_raw_buffer_load_b128(from, off, 0, 0), 16);
#endif
}

// BYTES bytes (1 to 4 N) wherever they begin.
template <int BYTES, int N>
__device__ __forceinline__ void words_at(const void* from, unsigned (&to)[N]) {
  if constexpr (BYTES < 4) to[N - 1] = 0;
  __builtin_memcpy(to, from, BYTES);
}

// The low end of a number of N words without its first n units of BITS bits,
// zeros behind.
template <int BITS, int N>
__device__ __forceinline__ void without(unsigned (&w)[N], int n) {
  typedef unsigned __int128 wide;
  wide v = 0;
  __builtin_memcpy(&v, w, 4 * N);
  v = n * BITS < 128 ? v >> (n * BITS) : 0;
  __builtin_memcpy(w, &v, 4 * N);
}

// The result of row m and column n of group g over K k from the definition, sum
// of s (q - z) x in 64 bits, for sums that left FP32: (16 + q) x and (16 + z) x
// of an infinite activation are infinities whose difference is NaN, and those of
// a finite one from 2^123 on may leave FP32 where their difference would not.
// (Such a result alone pays for it, and NaN ends it: 33 rows, 4096 x 11008, 20.5
// us, 102 with one infinite activation, 21.1 with a NaN.  All others pay for the
// check: 64 rows 24.8 and 25.0 us without and with it; 64 experts of 2048 x 2048, 512
// rows, 46.2 and 46.4.)
template <bool BF, int GB>
__device__ __forceinline__ float defined(int g, int64_t m, int64_t n, int K) {
#if defined(__HIP_DEVICE_COMPILE__)
  // (The arguments are read once more: kept through the kernel's loops they
  // would cost some ten scalar registers that it does not have.)
  typedef const __attribute__((address_space(4))) MatmulArgs args;
  args* p = (args*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  const uint8_t* const codes = p->codes + g * p->stride_q + n * p->ldq;
  const uint16_t* const scales = static_cast<const uint16_t*>(p->scales) + g * p->stride_s + n * p->lds;
  const uint8_t* const zeros = p->zeros ? p->zeros + g * p->stride_z + n * p->ldz : nullptr;
  const uint16_t* const x = static_cast<const uint16_t*>(p->X) + m * p->ldx;
  double sum = 0.;
#pragma nounroll
  for (int k0 = 0; k0 < K; k0 += 32) {
    const double s = widen16<BF>(scales[k0 / GB]);
    const int z = zeros ? zeros[k0 / GB] : 8;
    const u32x4 w = *reinterpret_cast<const u32x4*>(codes + k0 / 2);
    auto term = [&](int u, uint16_t v) __attribute__((always_inline)) {
      sum = __builtin_fma(s * ((int)(w[u / 8] >> (4 * (u % 8)) & 15) - z), (double)widen16<BF>(v), sum);
    };
    if (k0 + 32 <= K) {
      uint16_t v[32];
      __builtin_memcpy(v, x + k0, sizeof(v));
#pragma unroll
      for (int u = 0; u < 32; ++u) term(u, v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < 32; ++u)
        if (k0 + u < K) term(u, x[k0 + u]);
    }
    if (sum != sum) break;
  }
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0) (see the results' loop)
  return (float)sum;
#else
  return 0.f;
#endif
}

template <bool BF, class S, Reads HOW>
__global__ void __launch_bounds__(64 * S::WAVES) matmul_few(MatmulArgs p, unsigned tiles, unsigned tiles_n) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef half_t<BF> T;
  constexpr int GB = S::GB, MB = S::MB, NB = S::NB, KW = S::KW, NW = S::NW, SPAN = S::SPAN, V = S::V, GROUPS = S::GROUPS;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S::LDS];
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), kw = wave / NW, nw = wave % NW;
  const int ng = (p.K + GB - 1) / GB, padded = (p.K + 31) / 32 * 32;
  const unsigned one = BF ? 0x3f803f80u : 0x3c003c00u;
  const h16x8_t ones = __builtin_bit_cast(h16x8_t, u32x4{one, one, one, one});
  uint8_t* const xs = lds + (S::SHARED ? kw * 2 * S::X_BYTES : 0);

  for (unsigned b = blockIdx.x; b < tiles; b += gridDim.x) {
    grouped::RowTile t;
    if (p.offsets) {
      t = grouped::RowTiles(p.offsets, p.G, p.T, p.fill, S::ROWS).find((int)(b / tiles_n));
      if (t.rows <= 0) break;  // (the grid holds the most tiles that offsets can give)
    } else {
      t.g = 0;
      t.row0 = (int)(b / tiles_n) * S::ROWS;
      t.rows = p.T - t.row0 < S::ROWS ? p.T - t.row0 : S::ROWS;
    }
    const int n0 = (int)(b % tiles_n) * S::COLS;
    const int K = t.g < 0 ? 0 : p.K;  // (rows of no group: a sum over no k)
    const int64_t g = t.g < 0 ? 0 : t.g;
    const int cols = p.N - n0 < S::COLS ? p.N - n0 : S::COLS;
    // Where this lane reads: WHOLE, byte offsets into the descriptors of the
    // tile's rows and columns (past their range: zeros); otherwise addresses,
    // with the last row and column in place of those past the end (their
    // results are not stored).
    const uint8_t* const codes0 = p.codes + g * p.stride_q + n0 * p.ldq;
    const uint16_t* const scales0 = static_cast<const uint16_t*>(p.scales) + g * p.stride_s + n0 * p.lds;
    // (Without zero points some of the codes in their place, not used.)
    const uint8_t* const zeros0 = p.zeros ? p.zeros + g * p.stride_z + n0 * p.ldz : codes0;
    const int64_t ldz = p.zeros ? p.ldz : p.ldq;
    const uint16_t* const x0 = static_cast<const uint16_t*>(p.X) + t.row0 * p.ldx;
    auto uniform = [](const void* at, int64_t bytes) __attribute__((always_inline)) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(at), 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t from_q = uniform(codes0, HOW == WHOLE && K > 0 ? (cols - 1) * p.ldq + padded / 2 : 0);
    const __amdgpu_buffer_rsrc_t from_s = uniform(scales0, HOW == WHOLE && K > 0 ? 2 * ((cols - 1) * p.lds + ng) : 0);
    const __amdgpu_buffer_rsrc_t from_z = uniform(zeros0, HOW == WHOLE && K > 0 && p.zeros ? (cols - 1) * p.ldz + ng : 0);
    const __amdgpu_buffer_rsrc_t from_x = uniform(x0, HOW == WHOLE && K > 0 ? 2 * ((t.rows - 1) * p.ldx + K) : 0);
    const unsigned kept = p.zeros ? ~0u : 0u, no_zeros = p.zeros ? 0u : 0x08080808u;
    int64_t col[NB];
    unsigned q_at[NB], s_at[NB], z_at[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int c = 16 * (NB * nw + j) + r;
      col[j] = HOW == WHOLE || c < cols ? c : cols - 1;
      q_at[j] = (unsigned)(col[j] * p.ldq) + (HOW == WHOLE ? 16 * q : 0);
      s_at[j] = (unsigned)(2 * col[j] * p.lds);
      z_at[j] = (unsigned)(col[j] * ldz);
    }
    // Piece i of X: its row, its k from the span's first on, its place in LDS.
    int row[S::XL], xk[S::XL], to[S::XL];
    unsigned x_at[S::XL];
#pragma unroll
    for (int i = 0; i < S::XL; ++i) {
      const int piece = 64 * (i * NW + nw) + l;
      const int m = S::SHARED ? piece / (SPAN / 8) : 16 * (i % MB) + r;
      const int c = S::SHARED ? piece % (SPAN / 8) : S::chunk(i / MB, q);
      row[i] = HOW == WHOLE || m < t.rows ? m : t.rows - 1;
      xk[i] = 8 * c;
      x_at[i] = 2 * (unsigned)(row[i] * (int)p.ldx) + (HOW == WHOLE ? 16 * c : 0);
      to[i] = S::x_byte(m, c);
    }

    // The span at k0 (uniform; from K on, something that does not count).  WHOLE
    // and SPANS have no branches: at one, the compiler would wait for loads that
    // are on their way.  SPANS reads from before the end of a row what would
    // lie past it, and moves it down (`trim`) where it is used.
    auto load = [&](int k0, Codes<S>& c) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if constexpr (HOW == WHOLE) {
          // (One uniform choice: past K an offset out of every range.)
          const unsigned q0 = k0 < K ? k0 / 2 : OOB, s0 = k0 < K ? 2 * (k0 / GB) : OOB, z0 = k0 < K ? k0 / GB : OOB;
#pragma unroll
          for (int h = 0; h < SPAN / 128; ++h) buffer_words<4>(from_q, q_at[j] + q0 + 64 * h, c.w[j][h]);
          buffer_words<(GROUPS + 1) / 2, 2 * GROUPS>(from_s, s_at[j] + s0, c.s[j]);
          buffer_words<(GROUPS + 3) / 4, GROUPS>(from_z, z_at[j] + z0, c.z[j]);
        } else if constexpr (HOW == SPANS) {
#pragma unroll
          for (int h = 0; h < SPAN / 128; ++h) {
            const int k = k0 + 128 * h + 32 * q;  // (the lane's piece is a whole 32 k, all of it there or none)
            const unsigned off = q_at[j] + (unsigned)grouped::code_byte(k, padded);
            __builtin_memcpy(c.w[j][h], __builtin_assume_aligned(codes0 + off, 16), 16);
          }
          const int i = grouped::piece_start(k0 / GB, ng, GROUPS);
          words_at<2 * GROUPS>((const uint8_t*)scales0 + (s_at[j] + (unsigned)(2 * i)), c.s[j]);
          words_at<GROUPS>(zeros0 + (z_at[j] + (unsigned)i), c.z[j]);
        } else if (k0 < K) {
#pragma unroll
          for (int h = 0; h < SPAN / 128; ++h) {
            const int at = grouped::code_byte(k0 + 128 * h + 32 * q, padded);
            __builtin_memcpy(c.w[j][h], __builtin_assume_aligned(codes0 + col[j] * p.ldq + at, 16), 16);
          }
#pragma unroll
          for (int h = 0; h < GROUPS; ++h) {
            const int i = grouped::piece_start(k0 / GB + h, ng, 1);
            c.s[j][h / 2] = (h % 2 ? c.s[j][h / 2] : 0u) | (unsigned)scales0[col[j] * p.lds + i] << (16 * (h % 2));
            c.z[j][h / 4] = (h % 4 ? c.z[j][h / 4] : 0u) | (p.zeros ? (unsigned)zeros0[col[j] * p.ldz + i] : 0u) << (8 * (h % 4));
          }
        }
      }
    };
    const bool pieces = HOW == SPANS || (HOW == ANY && p.K >= 8 && p.ldx < kFar);
    auto load_x = [&](int k0, u32x4 (&xv)[S::XL]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < S::XL; ++i) {
        if constexpr (HOW == WHOLE) {
          const unsigned off = k0 + xk[i] < K ? x_at[i] + 2 * k0 : OOB;
          buffer_words<4>(from_x, off, reinterpret_cast<unsigned(&)[4]>(xv[i]));
        } else if (pieces) {
          const int k = grouped::piece_start(k0 + xk[i], p.K, 8);  // (K may be 0)
          __builtin_memcpy(&xv[i], (const uint8_t*)x0 + (x_at[i] + (unsigned)(2 * k)), 16);
        } else {
          uint16_t e[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) e[u] = k0 + xk[i] + u < K ? x0[row[i] * p.ldx + k0 + xk[i] + u] : (uint16_t)0;
          __builtin_memcpy(&xv[i], e, 16);
        }
      }
    };
    auto trim_x = [&](int k0, u32x4 (&xv)[S::XL]) __attribute__((always_inline)) {
      if (!pieces || k0 + SPAN <= K) return;
#pragma unroll
      for (int i = 0; i < S::XL; ++i) {
        const int past = k0 + xk[i] - (K - 8);
        without<16>(reinterpret_cast<unsigned(&)[4]>(xv[i]), past > 0 ? past : 0);
      }
    };
    auto trim_scales = [&](int k0, Codes<S>& c) __attribute__((always_inline)) {
      const int past = k0 / GB - (ng - GROUPS);
      if (HOW != SPANS || GROUPS == 1 || past <= 0) return;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        without<16>(c.s[j], past);
        without<8>(c.z[j], past);
      }
    };
    auto store_x = [&](uint8_t* to_span, const u32x4 (&xv)[S::XL]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < S::XL; ++i) *reinterpret_cast<u32x4*>(to_span + to[i]) = reorder(xv[i]);
    };
    // LDS writes of the waves of one span are done (global loads may be on
    // their way: __syncthreads would wait for them).
    auto barrier = []() __attribute__((always_inline)) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    f32x4 acc[NB][MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    // A span's products; X from LDS or (not SHARED) from the lane's pieces.
    auto multiply = [&](int k0, Codes<S>& c, const uint8_t* xb) __attribute__((always_inline)) {
      if constexpr (GB < 128) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int h = 0; h < SPAN / 128; ++h) exchange(c.w[j][h]);
      }
      if constexpr (!S::SHARED) trim_x(k0, c.x);
      trim_scales(k0, c);
#pragma unroll
      for (int h = 0; h < GROUPS; ++h) {
        if (k0 / GB + h >= ng) break;
        h16x8_t xo[V][MB];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int i = 0; i < MB; ++i)
            if constexpr (S::SHARED)
              xo[v][i] = *reinterpret_cast<const h16x8_t*>(xb + S::x_byte(16 * i + r, S::chunk(h * V + v, q)));
            else
              xo[v][i] = __builtin_bit_cast(h16x8_t, reorder(c.x[(h * V + v) * MB + i]));
        f32x4 part[NB][MB], sx[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          sx[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < NB; ++j) part[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int i = 0; i < MB; ++i) sx[i] = mfma16<BF>(xo[v][i], ones, sx[i]);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const h16x8_t wv = __builtin_bit_cast(h16x8_t, widen<BF>(c.w[j][(h * V + v) / 4][(h * V + v) % 4]));
#pragma unroll
            for (int i = 0; i < MB; ++i) part[j][i] = mfma16<BF>(xo[v][i], wv, part[j][i]);
          }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const float s = widen16<BF>((unsigned short)(c.s[j][h / 2] >> (16 * (h % 2))));
          const float z = -16.f - (float)((c.z[j][h / 4] & kept | no_zeros) >> (8 * (h % 4)) & 255);
#pragma unroll
          for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[j][i][e] = __builtin_fmaf(s, __builtin_fmaf(z, sx[i][e], part[j][i][e]), acc[j][i][e]);
        }
      }
    };

    // Wave row kw takes spans kw, kw + KW, ..., each column of tiles from another
    // of them on (at one time the rows of all codes would be read at one offset, from
    // few of the memory's channels); all that DEPTH spans need is on its way in
    // registers (loads return in order, so what is asked for late would hold up
    // what was asked for early).  SHARED X goes on into one of two places in
    // LDS, a span ahead; then every wave takes part in every barrier.
    constexpr int DEPTH = S::SHARED && S::WAVES == 8 ? 4 : 2;  // (16 waves hide as much with half the registers)
    Codes<S> ring[DEPTH];
    const int spans = ((K + SPAN - 1) / SPAN + KW - 1) / KW;
    const int past = grouped::past_spans<SPAN>(K);
    const int turn = spans > 0 ? (int)(b % tiles_n % (unsigned)spans) : 0;
    auto at = [&](int i) __attribute__((always_inline)) { return grouped::span_start<KW, SPAN>(i, spans, turn, kw, past); };
    // (In the order of the spans everywhere: the waits count on it.)
    auto fetch = [&](int i, Codes<S>& c) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      load(at(i), c);
      load_x(at(i), c.x);
      __builtin_amdgcn_sched_barrier(0);
    };
    each<DEPTH>([&](auto D) __attribute__((always_inline)) { fetch(decltype(D)::value, ring[decltype(D)::value]); });
    if constexpr (S::SHARED) {
      barrier();  // (the tile before has been read)
      trim_x(at(0), ring[0].x);
      store_x(xs, ring[0].x);
    }
    auto span = [&](int i, auto D) __attribute__((always_inline)) {
      constexpr int d = decltype(D)::value;
      if constexpr (S::SHARED) {
        barrier();  // this span's X has been written, the place of the next one's read
        trim_x(at(i + 1), ring[(d + 1) % DEPTH].x);
        store_x(xs + (d + 1) % 2 * S::X_BYTES, ring[(d + 1) % DEPTH].x);
      }
      if (at(i) < K) multiply(at(i), ring[d], xs + d % 2 * S::X_BYTES);
      fetch(i + DEPTH, ring[d]);
    };
    for (int i = 0; i < spans; i += DEPTH) {
      span(i, std::integral_constant<int, 0>{});
      if (i + 1 >= spans) break;
      span(i + 1, std::integral_constant<int, 1>{});
      if constexpr (DEPTH == 4) {
        if (i + 2 >= spans) break;
        span(i + 2, std::integral_constant<int, 2>{});
        if (i + 3 >= spans) break;
        span(i + 3, std::integral_constant<int, 3>{});
      }
    }

    // Register e of lane l: row 16i + 4q + e, column 16j + r.
    float* const sums = reinterpret_cast<float*>(lds);
    barrier();
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[(kw * S::ROWS + 16 * i + 4 * q + e) * S::COLS + 16 * (NB * nw + j) + r] = acc[j][i][e];
    barrier();
    // vmcnt(0): with loads on their way, these or those of `defined`, the compiler
    // waits in the loop, and so for every result's store (64 rows, 4096 x 11008:
    // 25.6 us, with this wait 25.0).
    __builtin_amdgcn_s_waitcnt(0x0f70);
    for (int i = tid; i < S::ROWS * S::COLS; i += 64 * S::WAVES) {
      const int m = i / S::COLS, col = i % S::COLS;
      if (m >= t.rows || n0 + col >= p.N) continue;
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < KW; ++u) v += sums[(u * S::ROWS + m) * S::COLS + col];
      if (!(__builtin_fabsf(v) < __builtin_inff())) v = defined<BF, GB>(t.g, t.row0 + m, n0 + col, p.K);
      static_cast<T*>(p.Y)[(t.row0 + m) * p.ldy + n0 + col] = (T)v;
    }
  }
#endif
}

// SPANS: there is a matrix, a row of which holds a whole span's scales and
// eight k, and a tile's rows and columns are within 31 bits of bytes.  WHOLE: X
// in aligned 16-byte pieces besides, a span's scales and zero points as one
// aligned load each, all of them there (a load that is partly past a
// descriptor's range gives zeros).  (WHOLE, as SPANS and as ANY, one wave along k:
// 4096 x 11008, groups of 64, 33 rows 22.0, 22.6 and 84 us; 64 rows, groups of 128
// 26.7, 27.5 and 57; 64 experts of 2048 x 2048, 512 rows 49, 56 and 69, groups of 32
// 59, 64 and 217.  K 4095, one row of 4096 columns: 11.0 us SPANS, 38 ANY; 16 rows,
// which begin on 2 bytes: 30.3 and 38.5, of K 4096 10.)
template <class S>
Reads reads_of(const MatmulArgs& a) {
  constexpr int64_t g = S::GROUPS;
  const int64_t ng = groups_of(a.K, S::GB);
  if (a.G == 0 || a.K < 8 || ng < g || a.ldx >= kFar || a.ldq >= kFar || a.lds >= kFar || a.ldz >= kFar) return ANY;
  const bool x = (uintptr_t)a.X % 16 == 0 && a.ldx % 8 == 0 && a.K % 8 == 0;
  const bool s = (uintptr_t)a.scales % (2 * g) == 0 && a.lds % g == 0 && (a.G <= 1 || a.stride_s % g == 0);
  const bool z = !a.zeros || ((uintptr_t)a.zeros % g == 0 && a.ldz % g == 0 && (a.G <= 1 || a.stride_z % g == 0));
  return x && s && z && ng % g == 0 ? WHOLE : SPANS;
}

int64_t tiles_of(const MatmulArgs& a, int64_t rows, int64_t cols) {
  const int64_t tiles_m = a.offsets ? grouped::most_tiles(a.T, a.G, a.fill, (int)rows) : (a.T + rows - 1) / rows;
  return tiles_m * ((a.N + cols - 1) / cols);
}

template <bool BF, class S, Reads HOW>
hipError_t start(const MatmulArgs& a, hipStream_t s) {
  const int64_t tiles = tiles_of(a, S::ROWS, S::COLS), tiles_n = ((int64_t)a.N + S::COLS - 1) / S::COLS;
  if (tiles <= 0) return hipSuccess;
  if (tiles >= 1ll << 31) return hipErrorInvalidConfiguration;  // (of a result that no memory holds)
  constexpr int64_t threads = 64 * S::WAVES, most = kMostItems / threads;
  hipLaunchKernelGGL((matmul_few<BF, S, HOW>), dim3((unsigned)(tiles < most ? tiles : most)), dim3((unsigned)threads), 0, s, a,
                     (unsigned)tiles, (unsigned)tiles_n);
  return hipGetLastError();
}

template <bool BF, int GB, int MB, Reads HOW>
hipError_t along(const MatmulArgs& a, int kw, hipStream_t s) {
  if constexpr (MB == 1) {
    if (kw == 8) return start<BF, Shape<GB, MB, 1, 8>, HOW>(a, s);
  }
  if (kw >= 4) return start<BF, Shape<GB, MB, 1, 4>, HOW>(a, s);
  // (12 KB of X do not split over eight waves along the columns: four, and four
  // along k.  M 33, 4096 x 11008: 19.0 us, 23.3 with two along k; with one or two
  // blocks of rows 16 waves gain nothing: M 1, 4096 x 4096, 9.0 us and 6.8 with 8.)
  if constexpr (MB == 3) return start<BF, Shape<GB, MB, 1, 4, 16>, HOW>(a, s);
  else return kw == 1 ? start<BF, Shape<GB, MB, 1, 1>, HOW>(a, s) : start<BF, Shape<GB, MB, 1, 2>, HOW>(a, s);
}

template <bool BF, int GB, int MB>
hipError_t on_rows(const MatmulArgs& a, int kw, hipStream_t s) {
  switch (reads_of<Shape<GB, MB, 1, 4>>(a)) {
    case WHOLE: return along<BF, GB, MB, WHOLE>(a, kw, s);
    case SPANS: return along<BF, GB, MB, SPANS>(a, kw, s);
    default: return start<BF, Shape<GB, 1, 1, 1>, ANY>(a, s);  // (a row is a span at most, but for far strides)
  }
}

}  // namespace

template <int DT, int GB>
hipError_t launch_few(const MatmulArgs& a, hipStream_t s) {
  constexpr bool BF = DT == GEMM_DTYPE_BF16;
  // The most waves along k whose tiles are no more than the CUs, one round of
  // them (4096 x 4096, one row: 8 waves along k, 256 tiles, 6.7 us; 4, 128 tiles,
  // 10.9.  4096 x 11008: 2, 172 tiles, 14.7 us; 4, 344 tiles, 19.9.  7105 x 8448, five
  // rows: 2, 132 tiles, 32 us; 4, 264 tiles, 47.)  Experts: tiles that are likely,
  // not those of the worst offsets.
  const int64_t rows = a.offsets && a.G > 0 ? ((int64_t)a.T + a.G - 1) / a.G : a.T;
  auto likely = [&](int64_t tile_rows, int64_t kw) {
    const int64_t m = a.offsets ? (a.T < a.G ? (int64_t)a.T : a.T / tile_rows + a.G / 2) : (a.T + tile_rows - 1) / tile_rows;
    return m * ((a.N + 16 * (8 / kw) - 1) / (16 * (8 / kw)));
  };
  auto along_k = [&](int64_t tile_rows) {
    int kw = 1;
    while (kw < 8 && likely(tile_rows, 2 * kw) <= 256) kw *= 2;
    return kw;
  };
  // More rows a tile read fewer codes and more of X at once (M 64: 4096 x 4096
  // 14.1 us on 32 rows, 18.9 on 64; 4096 x 11008 30.2 and 24.7).  48 and 64 rows,
  // dense: M 33, 40 and 48, 4096 x 6144 16.2, 15.4 and 15.7 us on 48 and 19.3, 18.8
  // and 19.2 on 64; 4096 x 11008 19.5, 19.5 and 19.8 against 24.2, 24.3 and 24.5; 4096
  // x 22016 36.9, 37.2 and 37.7 against 39.1, 39.2 and 39.6; groups of 32 alike.
  // Experts: their rows differ, so that tiles of 48 are half empty where 64 were,
  // only more of them: 1280 rows, 32 of 2048 x 2048, 66.4 and 64.9 us, groups of 32
  // 81.6 and 64.9; 384 rows evenly to 8 of 2048 x 4096 27.5 and 24.0 (but 288 rows
  // unevenly to 8 of 4096 x 4096 56.3 and 76.8).
  if (rows <= (a.offsets ? 16 : 32)) return on_rows<BF, GB, 1>(a, along_k(16), s);
  if (rows <= 32 || likely(64, 4) < 160) return on_rows<BF, GB, 2>(a, along_k(32), s);
  if (rows <= 48 && !a.offsets) return on_rows<BF, GB, 3>(a, along_k(48), s);
  return on_rows<BF, GB, 4>(a, along_k(64), s);
}

template hipError_t launch_few<W4_TYPE, W4_GROUP>(const MatmulArgs&, hipStream_t);

}  // namespace w4
}  // namespace gemm

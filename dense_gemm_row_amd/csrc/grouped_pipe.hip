// The pipelined kernels of the grouped products, for 16-bit operands of whole
// 16-byte pieces.  One file for every combination of GROUPED_TYPE (element
// type), GROUPED_OUT (the result's) and GROUPED_TILE (tile): compiled once for
// each.
#if !defined(GROUPED_TYPE) || !defined(GROUPED_OUT) || !defined(GROUPED_TILE)
#error "compiled once for every GROUPED_TYPE, GROUPED_OUT and GROUPED_TILE"
#endif

#include "grouped_internal.h"
#include "mx_pipe.h"

namespace gemm {
namespace grouped {
namespace {

using mx::IC;
using mx::OOB;
using mx::f32x4;
using mx::i32x2;
using mx::i32x4;

template <bool BF>
__device__ __forceinline__ void mfma_asm(f32x4& c, i32x4 a, i32x4 b) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (BF) mx::mfma_bf16_asm(c, a, b);
  else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
#endif
}

// A workgroup of four waves computes BM x BN results, each wave WM x WN of
// them in 16 x 16 blocks, 64 k per slice through two LDS stages.  Operands go
// to LDS with 16-byte LDS-direct copies as they lie in memory:
//  * ALONG (k contiguous: X; W given transposed): a row of 64 k is 128 bytes,
//    its 16-byte chunks XORed by (row / 2) % 8; an operand is one 16-byte read.
//  * ACROSS (rows contiguous, k down the rows: W; both of the gradient's): 64
//    rows of 2 BM (2 BN) bytes, chunks XORed by 4 (k % 4) + 2 (k / 8 % 2); an
//    operand is two transpose reads (in each group of 16 lanes, lane j gets
//    element j % 4 of the 8-byte pieces that lanes j / 4 + 4t point at).
// Lane group q takes k 32j + 8q .. + 7 of a slice in step j.  Rows and chunks
// past an operand's end are past their descriptor's range, or masked, and land
// in LDS as zeros: the last rows of a group's tile, the end of k, and for the
// gradient the end of the group's rows.
template <bool A_ACROSS_, bool B_ACROSS_, int BM_, int BN_, int WM_, int WN_, int NS_ = 2>
struct Tile {
  static constexpr bool A_ACROSS = A_ACROSS_, B_ACROSS = B_ACROSS_;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 64, NS = NS_;
  static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  static constexpr int MB = WM / 16, NB = WN / 16, NMMA = MB * NB;
  static constexpr int A_STAGE = BM * 2 * BK, B_STAGE = BN * 2 * BK;
  static constexpr int IA = A_STAGE / 1024 / NW, IB = B_STAGE / 1024 / NW, LPS = IA + IB;
  static_assert(NW == 4 && IA > 0 && IB > 0, "copies split over four waves");
  static_assert((!A_ACROSS || BM >= 128) && (!B_ACROSS || BN >= 128), "rows of at least 256 bytes (the chunk XOR)");
  __host__ __device__ static constexpr int along_byte(int row, int c) { return 128 * row + 16 * (c ^ (row / 2 % 8)); }
  __host__ __device__ static constexpr int across_swz(int k) { return (4 * (k % 4)) ^ (2 * (k / 8 % 2)); }
  __host__ __device__ static constexpr int across_byte(int width, int k, int n) {
    return 2 * width * k + 16 * (n / 8 ^ across_swz(k)) + 2 * (n % 8);
  }
  // Slots of a step's reads and of a slice's copies among its instructions.
  __host__ __device__ static constexpr int rd_slot(int f) { return f * NMMA / (MB + NB); }
  __host__ __device__ static constexpr int cp_slot(int c) { return (2 * c + 1) * NMMA / (2 * LPS); }
};

// Offsets of this lane's copies of one operand, from its descriptor's base.
// ALONG: `rows` rows exist; ACROSS: `rows` (a multiple of 8) of a k row do.
template <bool ACROSS, int WIDTH, int N>
struct Copies {
  unsigned off[N];
  int chunk[N];  // ALONG: 16-byte chunk of k
  __device__ __forceinline__ Copies(int wave, int l, int ld, int rows) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned at = 1024 * (4 * i + wave) + 16 * l;
      if constexpr (ACROSS) {
        const int k = at / (2 * WIDTH), c = (at % (2 * WIDTH) / 16) ^ ((4 * (k % 4)) ^ (2 * (k / 8 % 2)));
        off[i] = 8 * c < rows ? (unsigned)(2 * (k * ld + 8 * c)) : OOB;
        chunk[i] = 0;
      } else {
        const int row = at / 128;
        chunk[i] = (at % 128 / 16) ^ (row / 2 % 8);
        off[i] = row < rows ? (unsigned)(2 * (row * ld + 8 * chunk[i])) : OOB;
      }
    }
  }
};

// The descriptor of the slice of an operand from `base` (its first row at the
// slice's first k) on: `left` k remain (0 or less: nothing is in range and the
// stage gets zeros).  A slice's copies share it.
template <bool ACROSS>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t slice_range(const uint16_t* base, int ld, int rows, int left) {
  if constexpr (ACROSS) {
    const int n = left < 64 ? left : 64;
    return mx::make_rsrc(base, n > 0 ? 2 * ((n - 1) * ld + ((rows + 7) & ~7)) : 0);
  } else {
    return mx::make_rsrc(base, 0x7fffffff);
  }
}

// Copy i of a slice.
template <bool ACROSS, int WIDTH, int N>
__device__ __forceinline__ void copy_one(const Copies<ACROSS, WIDTH, N>& o, int i, __amdgpu_buffer_rsrc_t from, int left,
                                         uint8_t* stage, int wave) {
#if defined(__HIP_DEVICE_COMPILE__)
  mx::lds_void* to = (mx::lds_void*)(stage + 1024 * (4 * i + wave));
  const unsigned off = ACROSS || 8 * o.chunk[i] < left ? o.off[i] : OOB;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, to, 16, off, 0, 0, 0);
#endif
}

// The LDS stages, A and behind it B: arrays of their own, so that the compiler
// sees that copies into one do not touch what is read from another.
template <int NS>
struct Stages {
  uint8_t* at[NS];
};

// mx::loop_barrier, but for the last N copies, which need not have landed.
template <int N>
__device__ __forceinline__ void barrier_but() {
  static_assert(N < 64, "what the wait can count");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);  // vmcnt(N) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// acc[j][i], register e of lane l: row 16i + l%16, column 16j + 4(l/16) + e of
// the wave's share of A x B over K k; A has `rows` rows and B `cols` columns
// from the tile on.
template <bool BF, class S>
__device__ __forceinline__ void tile_sums(const Stages<S::NS>& lds, const uint16_t* A, int lda, int rows, const uint16_t* B, int ldb, int cols, int K,
                                          f32x4 (&acc)[S::NB][S::MB]) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int MB = S::MB, NB = S::NB, BK = S::BK, NS = S::NS;
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / S::WAVES_N) * S::WM, wn0 = (wave % S::WAVES_N) * S::WN;
  const Copies<S::A_ACROSS, S::BM, S::IA> ca(wave, l, lda, rows);
  const Copies<S::B_ACROSS, S::BN, S::IB> cb(wave, l, ldb, cols);
  // Fragment addresses: ALONG one a step (blocks are 2 KB apart), ACROSS one
  // a block (steps are 32 rows apart).
  int a_fb[S::A_ACROSS ? MB : 2], b_fb[S::B_ACROSS ? NB : 2];
  if constexpr (S::A_ACROSS) {
#pragma unroll
    for (int i = 0; i < MB; ++i) a_fb[i] = S::across_byte(S::BM, 8 * q + r / 4, wm0 + 16 * i + 4 * (r % 4));
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) a_fb[j] = S::along_byte(wm0 + r, 4 * j + q);
  }
  if constexpr (S::B_ACROSS) {
#pragma unroll
    for (int i = 0; i < NB; ++i) b_fb[i] = S::across_byte(S::BN, 8 * q + r / 4, wn0 + 16 * i + 4 * (r % 4));
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) b_fb[j] = S::along_byte(wn0 + r, 4 * j + q);
  }
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  mx::pin(acc);
  mx::mfma_guard();

  auto transposed = [](const uint8_t* p, int row) __attribute__((always_inline)) {
    const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx::lds_s16x4*)p));
    const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx::lds_s16x4*)(p + 4 * row)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
  };
  i32x4 fa[2][MB], fb[2][NB];
  // Operand f of step j from a stage: A's MB blocks, then B's NB.
  auto read = [&](const uint8_t* la, const uint8_t* lb, auto J, auto F) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value, f = decltype(F)::value;
    if constexpr (f < MB) {
      if constexpr (S::A_ACROSS) fa[j][f] = transposed(la + a_fb[f] + 32 * j * 2 * S::BM, 2 * S::BM);
      else fa[j][f] = *(const mx::lds_i32x4*)(la + a_fb[j] + 2048 * f);
    } else {
      constexpr int g = f - MB;
      if constexpr (S::B_ACROSS) fb[j][g] = transposed(lb + b_fb[g] + 32 * j * 2 * S::BN, 2 * S::BN);
      else fb[j][g] = *(const mx::lds_i32x4*)(lb + b_fb[j] + 2048 * g);
    }
  };
  auto range_a = [&](int k0) __attribute__((always_inline)) {
    return slice_range<S::A_ACROSS>(A + (S::A_ACROSS ? (int64_t)k0 * lda : (int64_t)k0), lda, rows, K - k0);
  };
  auto range_b = [&](int k0) __attribute__((always_inline)) {
    return slice_range<S::B_ACROSS>(B + (S::B_ACROSS ? (int64_t)k0 * ldb : (int64_t)k0), ldb, cols, K - k0);
  };
  auto copy = [&](__amdgpu_buffer_rsrc_t ra, __amdgpu_buffer_rsrc_t rb, int left, uint8_t* la, uint8_t* lb, auto C)
      __attribute__((always_inline)) {
    constexpr int c = decltype(C)::value;
    if constexpr (c < S::IA) copy_one(ca, c, ra, left, la, wave);
    else copy_one(cb, c - S::IA, rb, left, lb, wave);
  };
  // Step j: its instructions in a fixed order, with the other step's reads and
  // the copies between them.
  auto step = [&](auto J, auto&& rd, auto&& cp) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value;
    mx::static_for([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      mfma_asm<BF>(acc[i / MB][i % MB], fb[j][i / MB], fa[j][i % MB]);
      mx::static_for([&](auto F) __attribute__((always_inline)) {
        if constexpr (S::rd_slot(decltype(F)::value) == i) rd(F);
      }, std::make_integer_sequence<int, MB + NB>{});
      mx::static_for([&](auto C) __attribute__((always_inline)) {
        if constexpr (S::cp_slot(decltype(C)::value) == i) cp(C);
      }, std::make_integer_sequence<int, S::LPS>{});
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, S::NMMA>{});
  };
  // The slice at k0 in stage c: step 0 with step 1's reads; the next slice
  // has landed and every wave has read stage c; step 1 with the next stage's
  // reads and the copies of the slice NS further into stage c.
  auto slice = [&](auto C, int k0) __attribute__((always_inline)) {
    constexpr int c = decltype(C)::value;
    uint8_t *la = lds.at[c], *lb = la + S::A_STAGE, *na = lds.at[(c + 1) % NS], *nb = na + S::A_STAGE;
    step(IC<0>{}, [&](auto F) __attribute__((always_inline)) { read(la, lb, IC<1>{}, F); }, [](auto) {});
    const int next = k0 + NS * BK;
    const __amdgpu_buffer_rsrc_t ra = range_a(next), rb = range_b(next);
    barrier_but<(NS - 2) * S::LPS>();
    __builtin_amdgcn_sched_barrier(0);
    step(IC<1>{}, [&](auto F) __attribute__((always_inline)) { read(na, nb, IC<0>{}, F); },
         [&](auto Q) __attribute__((always_inline)) { copy(ra, rb, K - next, la, lb, Q); });
  };
  // (With no k at all the stages get zeros and the loop is not entered.)
  mx::static_for([&](auto N) __attribute__((always_inline)) {
    constexpr int n = decltype(N)::value;
    const __amdgpu_buffer_rsrc_t ra = range_a(n * BK), rb = range_b(n * BK);
    mx::static_for([&](auto Q) __attribute__((always_inline)) { copy(ra, rb, K - n * BK, lds.at[n], lds.at[n] + S::A_STAGE, Q); },
                   std::make_integer_sequence<int, S::LPS>{});
  }, std::make_integer_sequence<int, NS>{});
  barrier_but<(NS - 1) * S::LPS>();
  mx::static_for([&](auto F) __attribute__((always_inline)) { read(lds.at[0], lds.at[0] + S::A_STAGE, IC<0>{}, F); },
                 std::make_integer_sequence<int, MB + NB>{});
  mx::mfma_guard();
  // (Slices past the end are zeros.  No way out of the loop's middle: at its
  // start the compiler would wait for copies that are on their way.)
  int64_t k0 = 0;
  if constexpr (NS == 4) {
    for (; k0 + 2 * BK < K; k0 += NS * BK) {
      slice(IC<0>{}, (int)k0);
      slice(IC<1>{}, (int)k0 + BK);
      slice(IC<2>{}, (int)k0 + 2 * BK);
      slice(IC<3>{}, (int)k0 + 3 * BK);
    }
  }
  for (; k0 < K; k0 += 2 * BK) {
    slice(IC<0>{}, (int)k0);
    slice(IC<1>{}, (int)k0 + BK);
  }
  __builtin_amdgcn_s_waitcnt(0x0070);
#endif
}

// Stores of one 16-row block row of a wave's share, m0 its first row, to rows of
// `ld` bytes, 16-byte aligned and whole: as mx::store_block_row, whose stores
// cover 64 bytes of 16 rows each, but lanes r and r + 8 of 16 exchange halves, so
// that a store covers 128 bytes, a cache line, of eight rows.  (By 64 bytes HBM
// was written 1.45 times the result's bytes.  16384 rows, 8 groups, 4096 x 4096
// bfloat16: 478 us by 64 bytes, 460 by lines; 64 groups, 1024 x 2048: 128 and 121.)
template <int CT, int NB>
__device__ __forceinline__ void store_lines(const void* C, unsigned ld, int m0, int rows, int cols, const f32x4 (&v)[NB]) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename mx::TypeOf<CT>::type T;
  constexpr unsigned es = sizeof(T);
  constexpr int STEP = es == 4 ? 2 : 4;  // blocks of a line
  static_assert(NB % STEP == 0, "whole lines");
  const int l = threadIdx.x & 63, r = l % 16, q = l / 16, half = r / 8, m = m0 + r % 8;
  const __amdgpu_buffer_rsrc_t to = mx::make_rsrc(C, 0x7fffffff);
  const unsigned row0 = m < rows ? (unsigned)m * ld : OOB, row1 = m + 8 < rows ? (unsigned)(m + 8) * ld : OOB;
#pragma unroll
  for (int nb = 0; nb < NB; nb += STEP) {
    i32x4 part[2], line[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (es == 4) {
        part[h] = __builtin_bit_cast(i32x4, v[nb + h]);
      } else {
        typedef T t2 __attribute__((ext_vector_type(2)));
        unsigned x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = __builtin_bit_cast(unsigned, t2{(T)v[nb + 2 * h][2 * i], (T)v[nb + 2 * h][2 * i + 1]});
          y[i] = __builtin_bit_cast(unsigned, t2{(T)v[nb + 2 * h + 1][2 * i], (T)v[nb + 2 * h + 1][2 * i + 1]});
        }
        const i32x2 s0 = __builtin_bit_cast(i32x2, __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false));
        const i32x2 s1 = __builtin_bit_cast(i32x2, __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false));
        part[h] = i32x4{s0[0], s1[0], s0[1], s1[1]};
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // (row_ror:8, written to lanes 8 .. 15 and to lanes 0 .. 7)
      line[0][e] = __builtin_amdgcn_update_dpp(part[0][e], part[1][e], 0x128, 0xf, 0xc, false);
      line[1][e] = __builtin_amdgcn_update_dpp(part[1][e], part[0][e], 0x128, 0xf, 0x3, false);
    }
    const int n = es == 4 ? 16 * (nb + half) + 4 * q : 16 * (nb + 2 * half + q % 2) + 8 * (q / 2);
    __builtin_amdgcn_raw_buffer_store_b128(line[0], to, n < cols ? row0 + n * es : OOB, 0, 2);
    __builtin_amdgcn_raw_buffer_store_b128(line[1], to, n < cols ? row1 + n * es : OOB, 0, 2);
  }
#endif
}

// The same for FP32 through `buf` in LDS, this wave's own: stores of whole rows of
// the share.  (Gradient of 16384 rows, 8 groups, 4096 x 4096: 520 us by 64 bytes, 505
// by lines, 1.33 times the bytes written, and 487 by rows, 1.09 times.)
template <class S>
__device__ __forceinline__ void store_rows(const void* C, unsigned ld, int m0, int rows, int cols, const f32x4 (&v)[S::NB],
                                           uint8_t* buf) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ROW = 4 * S::WN + 16, LANES = S::WN / 4, PER = 64 / LANES;  // (16 rows' writes meet distinct banks)
  const int l = threadIdx.x & 63, r = l % 16, q = l / 16, n = 4 * (l % LANES);
  const __amdgpu_buffer_rsrc_t to = mx::make_rsrc(C, 0x7fffffff);
#pragma unroll
  for (int j = 0; j < S::NB; ++j) *(mx::lds_i32x4*)(buf + ROW * r + 64 * j + 16 * q) = __builtin_bit_cast(i32x4, v[j]);
#pragma unroll
  for (int k = 0; k < 16 / PER; ++k) {
    const int row = PER * k + l / LANES, m = m0 + row;
    const i32x4 line = *(const mx::lds_i32x4*)(buf + ROW * row + 4 * n);
    __builtin_amdgcn_raw_buffer_store_b128(line, to, m < rows && n < cols ? (unsigned)m * ld + 4 * n : OOB, 0, 2);
  }
#endif
}

// Stores the wave's share (see tile_sums) to C, its first element, of which
// `rows` x `cols` exist.  EPI: v = alpha v + beta old.
template <int CT, class S, bool VEC, bool EPI>
__device__ __forceinline__ void store(const void* C, int64_t ldc, int rows, int cols, f32x4 (&acc)[S::NB][S::MB], float alpha,
                                      float beta, [[maybe_unused]] uint8_t* buf) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr unsigned es = CT == GEMM_DTYPE_F32 ? 4 : 2;
  const int l = threadIdx.x & 63, r = l % 16, q = l / 16;
#pragma unroll
  for (int i = 0; i < S::MB; ++i) {
    const int m = 16 * i + r;
    const unsigned row = m < rows ? (unsigned)m * (unsigned)(ldc * es) : OOB;
    f32x4 v[S::NB];
#pragma unroll
    for (int j = 0; j < S::NB; ++j) v[j] = acc[j][i];
    if constexpr (EPI) {
      f32x4 old[S::NB];
#pragma unroll
      for (int j = 0; j < S::NB; ++j) old[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (beta != 0.f) mx::load_block_row<CT, S::NB, VEC>(C, row, cols, old, q);
#pragma unroll
      for (int j = 0; j < S::NB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[j][e] *= alpha;
          if (beta != 0.f) v[j][e] = __builtin_fmaf(beta, old[j][e], v[j][e]);
        }
    }
    if constexpr (VEC && es == 4) store_rows<S>(C, (unsigned)(ldc * es), 16 * i, rows, cols, v, buf);
    else if constexpr (VEC) store_lines<CT, S::NB>(C, (unsigned)(ldc * es), 16 * i, rows, cols, v);
    else mx::store_block_row<CT, S::NB, false>(C, row, cols, v, q);
    __builtin_amdgcn_sched_barrier(0);  // (one block row's values in registers at a time)
  }
#endif
}

// The same to rows that begin anywhere, all of the share's columns inside: four
// values a store, which needs no alignment.  (1531 rows, 16 groups, 1000 x 1337 to
// FP32: 19.7 us, 24.2 by element.)
template <int CT, class S>
__device__ __forceinline__ void store_inside(void* C, int64_t ldc, int rows, f32x4 (&acc)[S::NB][S::MB]) {
  typedef typename mx::TypeOf<CT>::type T;
  const int l = threadIdx.x & 63, r = l % 16, q = l / 16;
  T* at = static_cast<T*>(C) + r * ldc + 4 * q;
#pragma unroll
  for (int i = 0; i < S::MB; ++i) {
    if (16 * i + r < rows) {
#pragma unroll
      for (int j = 0; j < S::NB; ++j) {
        const T e[4] = {(T)acc[j][i][0], (T)acc[j][i][1], (T)acc[j][i][2], (T)acc[j][i][3]};
        __builtin_memcpy(at + 16 * i * ldc + 16 * j, e, sizeof(e));
      }
    }
  }
}

// vec: rows of the result are 16-byte aligned and whole.
template <int CT, class S, bool EPI>
__device__ __forceinline__ void finish(void* C, int64_t ldc, int rows, int cols, f32x4 (&acc)[S::NB][S::MB], int vec, float alpha,
                                       float beta, const Stages<S::NS>& lds) {
  mx::mfma_guard();
  mx::pin(acc);  // (read after the guard only)
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm0 = (wave / S::WAVES_N) * S::WM, wn0 = (wave % S::WAVES_N) * S::WN;
  void* at = static_cast<typename mx::TypeOf<CT>::type*>(C) + wm0 * ldc + wn0;
  uint8_t* buf = lds.at[0] + wave * 16 * (4 * S::WN + 16);
  static_assert(S::NW * 16 * (4 * S::WN + 16) <= S::A_STAGE + S::B_STAGE, "a wave's block row");
  if (CT == GEMM_DTYPE_F32 && vec) __syncthreads();  // (every wave has read its operands)
  if (vec) store<CT, S, true, EPI>(at, ldc, rows - wm0, cols - wn0, acc, alpha, beta, buf);
  else if (!EPI && cols - wn0 >= S::WN) store_inside<CT, S>(at, ldc, rows - wm0, acc);
  else store<CT, S, false, EPI>(at, ldc, rows - wm0, cols - wn0, acc, alpha, beta, buf);
}

#define LDS_STAGES(S, lds) \
  constexpr int kStage = S::A_STAGE + S::B_STAGE, kMore = S::NS > 2 ? kStage : 16; \
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage], s1[kStage], s2[kMore], s3[kMore]; \
  Stages<S::NS> lds; \
  if constexpr (S::NS > 2) lds = {{s0, s1, s2, s3}}; \
  else lds = {{s0, s1}};

// One tile of the product: its rows and columns on a workgroup of shape S.
template <int DT, int CT, class S>
__device__ __forceinline__ void product_tile(const MatmulArgs& p, const Stages<S::NS>& lds, int g, int row0, int rows, int n0, int vec) {
  const uint16_t* X = static_cast<const uint16_t*>(p.X) + row0 * p.ldx;
  const uint16_t* W = static_cast<const uint16_t*>(p.W) + (g < 0 ? 0 : g) * p.stride_w + (S::B_ACROSS ? n0 : n0 * p.ldw);
  f32x4 acc[S::NB][S::MB];
  // (Rows of no group: a sum over no k.)
  tile_sums<DT == GEMM_DTYPE_BF16, S>(lds, X, (int)p.ldx, rows, W, (int)p.ldw, p.N - n0, g < 0 ? 0 : p.K, acc);
  finish<CT, S, false>(static_cast<typename mx::TypeOf<CT>::type*>(p.Y) + row0 * p.ldy + n0, p.ldy, rows, p.N - n0, acc, vec, 1.f,
                       0.f, lds);
}

// Tiles of 256 rows: those of no more than 128 rows, the last of most groups,
// and the last tiles of the grid where they would occupy no more than half of
// the CUs, each as two workgroups, run on 128 x 256 (HALF): about half the
// time.  kCus workgroups fill the GPU, one a CU.
template <int DT, int CT, class S, class HALF>
__global__ void __launch_bounds__(64 * S::NW) matmul_pipe(MatmulArgs p, int tiles_n, int vec) {
#if defined(__HIP_DEVICE_COMPILE__)
  LDS_STAGES(S, lds);
  constexpr bool HALVES = S::BM == 256;
  // The grid holds the most tiles that offsets can give; those that there are
  // are dealt to the XCDs in equal runs.
  const RowTiles all(p.offsets, p.G, p.T, p.fill, S::BM);
  const int tiles_m = all.count, tiles = tiles_m * tiles_n;
  const int last = HALVES && tiles % kCus <= kCus / 2 ? tiles % kCus : 0, first = tiles - last;
  int b = blockIdx.x, half = 0;
  if (b >= first + 2 * last) return;
  if (b < first) {
    const int x = b % kXcds, q = first / kXcds, r = first % kXcds;  // (as tile_of_block)
    b = x * q + (x < r ? x : r) + b / kXcds;
  } else {
    half = 1 + (b - first) % 2;
    b = first + (b - first) / 2;
  }
  int tm, tn;
  tile_of_block(b, TileMap{tiles_m, tiles_n, GEMM_ORDER_GROUPED, 4, kXcds}, tm, tn);
  const RowTile t = all.find(tm);
  // (Said to be uniform: the descriptors have to be in scalar registers.)
  const int g = __builtin_amdgcn_readfirstlane(t.g), n0 = __builtin_amdgcn_readfirstlane(tn * S::BN);
  int row0 = __builtin_amdgcn_readfirstlane(t.row0), rows = __builtin_amdgcn_readfirstlane(t.rows);
  if constexpr (HALVES) {
    if (half == 1) rows = rows < HALF::BM ? rows : HALF::BM;
    if (half == 2) {
      row0 += HALF::BM;
      rows -= HALF::BM;
      if (rows <= 0) return;
    }
    if (rows <= HALF::BM) return product_tile<DT, CT, HALF>(p, lds, g, row0, rows, n0, vec);
  }
  product_tile<DT, CT, S>(p, lds, g, row0, rows, n0, vec);
#endif
}

template <int DT, int CT, class S, bool EPI>
__global__ void __launch_bounds__(64 * S::NW) wgrad_pipe(WgradArgs p, int tiles_k, int tiles_n, int vec) {
#if defined(__HIP_DEVICE_COMPILE__)
  LDS_STAGES(S, lds);
  // One group after another, the longest first (they differ in rows, so the last
  // tiles should be the shortest), each dealt to all XCDs.
  const int each = tiles_k * tiles_n;
  const int rank = __builtin_amdgcn_readfirstlane((int)blockIdx.x / each);
  int tm, tn;
  tile_of_block((int)blockIdx.x - rank * each, TileMap{tiles_k, tiles_n, GEMM_ORDER_XCD, 4, kXcds}, tm, tn);
  const int m0 = __builtin_amdgcn_readfirstlane(tm * S::BM), n0 = __builtin_amdgcn_readfirstlane(tn * S::BN);
  int g, first, end;
  ranked_group(p.offsets, p.T, p.G, rank, g, first, end);
  g = __builtin_amdgcn_readfirstlane(g);
  first = __builtin_amdgcn_readfirstlane(first);
  end = __builtin_amdgcn_readfirstlane(end);
  const uint16_t* X = static_cast<const uint16_t*>(p.X) + first * p.ldx + m0;
  const uint16_t* dY = static_cast<const uint16_t*>(p.dY) + first * p.ldy + n0;
  f32x4 acc[S::NB][S::MB];
  tile_sums<DT == GEMM_DTYPE_BF16, S>(lds, X, (int)p.ldx, p.K - m0, dY, (int)p.ldy, p.N - n0, end - first, acc);
  finish<CT, S, EPI>(static_cast<typename mx::TypeOf<CT>::type*>(p.dW) + g * p.stride_w + m0 * p.ldw + n0, p.ldw, p.K - m0,
                     p.N - n0, acc, vec, p.alpha, p.beta, lds);
#endif
}

bool rows_whole(const void* C, int64_t ld, int64_t stride, int64_t cols, int64_t es) {
  return (uintptr_t)C % 16 == 0 && ld * es % 16 == 0 && stride * es % 16 == 0 && cols * es % 16 == 0;
}

}  // namespace

template <bool A, bool B, int SIDE, int NS = 2>
using TileOf = Tile<A, B, SIDE, SIDE, SIDE / 2, SIDE / 2, NS>;

template <int DT, int CT, int SIDE, int NS>
hipError_t on_stages(const MatmulArgs& a, hipStream_t s) {
  typedef TileOf<false, true, SIDE, NS> S;
  typedef TileOf<false, false, SIDE, NS> St;
  typedef Tile<false, true, 128, 256, 64, 128> H;
  typedef Tile<false, false, 128, 256, 64, 128> Ht;
  const int vec = rows_whole(a.Y, a.ldy, 0, a.N, CT == GEMM_DTYPE_F32 ? 4 : 2);
  const int64_t tiles_n = ((int64_t)a.N + S::BN - 1) / S::BN;
  const int64_t tiles = most_tiles(a.T, a.G, a.fill, S::BM) * tiles_n;
  if (tiles == 0) return hipSuccess;
  // (Up to kCus / 2 tiles are two workgroups.)
  const dim3 grid((unsigned)(tiles + (SIDE == 256 ? kCus / 2 : 0))), block(64 * S::NW);
  if (a.trans_w) hipLaunchKernelGGL((matmul_pipe<DT, CT, St, Ht>), grid, block, 0, s, a, (int)tiles_n, vec);
  else hipLaunchKernelGGL((matmul_pipe<DT, CT, S, H>), grid, block, 0, s, a, (int)tiles_n, vec);
  return hipGetLastError();
}

template <int DT, int CT, int SIDE, int NS>
hipError_t on_stages(const WgradArgs& a, hipStream_t s) {
  typedef TileOf<true, true, SIDE, NS> S;
  const int vec = rows_whole(a.dW, a.ldw, a.G > 1 ? a.stride_w : 0, a.N, CT == GEMM_DTYPE_F32 ? 4 : 2);
  const int64_t tiles_k = ((int64_t)a.K + S::BM - 1) / S::BM, tiles_n = ((int64_t)a.N + S::BN - 1) / S::BN;
  const dim3 grid((unsigned)(a.G * tiles_k * tiles_n)), block(64 * S::NW);
  if (grid.x == 0) return hipSuccess;
  if (a.alpha != 1.f || a.beta != 0.f)
    hipLaunchKernelGGL((wgrad_pipe<DT, CT, S, true>), grid, block, 0, s, a, (int)tiles_k, (int)tiles_n, vec);
  else
    hipLaunchKernelGGL((wgrad_pipe<DT, CT, S, false>), grid, block, 0, s, a, (int)tiles_k, (int)tiles_n, vec);
  return hipGetLastError();
}

template <int DT, int CT, int SIDE>
hipError_t launch_pipe(const MatmulArgs& a, hipStream_t s) {
  if constexpr (SIDE == 128) {
    if (alone(a)) return on_stages<DT, CT, SIDE, 4>(a, s);
  }
  return on_stages<DT, CT, SIDE, 2>(a, s);
}
template hipError_t launch_pipe<GROUPED_TYPE, GROUPED_OUT, GROUPED_TILE>(const MatmulArgs&, hipStream_t);

template <int DT, int CT, int SIDE>
hipError_t launch_pipe(const WgradArgs& a, hipStream_t s) {
  if constexpr (SIDE == 128) {
    if (alone(a)) return on_stages<DT, CT, SIDE, 4>(a, s);
  }
  return on_stages<DT, CT, SIDE, 2>(a, s);
}
template hipError_t launch_pipe<GROUPED_TYPE, GROUPED_OUT, GROUPED_TILE>(const WgradArgs&, hipStream_t);

}  // namespace grouped
}  // namespace gemm

// Product of two E2M1 (MXFP4) matrices, C = act(alpha A Bt^T + beta C + bias)
// (include/gemm_mx.h), on v_mfma_scale_f32_16x16x128_f8f6f4.
//
// The instruction multiplies 128 k values of 16 rows by 16 columns: lane l
// holds row l%16's 32 values of k block l/16 (16 bytes of codes) and that
// block's scale byte, which is exactly the storage format, so codes and
// scales go from memory to the matrix core without a conversion.  The
// operands are swapped (the result is C^T's block): register i of lane l is
// then C[l%16][4(l/16) + i], four consecutive columns of one row.
#include "mx_pipe.h"

namespace gemm {
namespace mx {
namespace {

constexpr int FP4 = 4;  // operand format field

__device__ __forceinline__ f32x4 mfma_fp4(i32x4 a, int sa, i32x4 b, int sb, f32x4 c) {
  const i32x8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, FP4, FP4, 0, sa, 0, sb);
}

// Columns n .. n+3 of row m from their sums (n < N; the row has N columns).
template <int DT>
__device__ __forceinline__ void store4(const MatmulArgs& p, int64_t m, int64_t n, f32x4 acc) {
  typedef typename TypeOf<DT>::type T;
  typedef T t4 __attribute__((ext_vector_type(4)));
  T* c = static_cast<T*>(p.C) + m * p.ldc + n;
  const bool whole = n + 4 <= p.N && ((uintptr_t)c & (sizeof(t4) - 1)) == 0;
  if (p.epi.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= p.N) break;
      const float old = p.epi.beta != 0.f ? (float)c[i] : 0.f;
      acc[i] = epi_value(p.epi, acc[i], old, p.epi.bias ? p.epi.bias[n + i] : 0.f);
    }
  }
  if (whole) {
    *reinterpret_cast<t4*>(c) = t4{(T)acc[0], (T)acc[1], (T)acc[2], (T)acc[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) c[i] = (T)acc[i];
  }
}

// A workgroup of W waves computes MT*16 rows x NT*16 columns; the waves
// take turns along k, U instructions' depth (U * 128) each, straight from
// memory, and their sums meet in LDS in wave order.  Rows and columns past
// the matrix repeat its last one and are not stored; blocks past the last
// are zeros.
template <int DT, int MT, int NT, int W, int U>
__global__ void __launch_bounds__(64 * W)
matmul_direct(MatmulArgs p, int tiles_n, int64_t tiles) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  __shared__ __attribute__((aligned(16))) float sums[W][BM][BN];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane % 16, q = lane / 16;
  const int nb = (p.K + BLOCK - 1) / BLOCK;
  const int steps = (nb + 3) / 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m0 = tile / tiles_n * BM, n0 = tile % tiles_n * BN;
    const uint8_t *ac[MT], *as[MT], *bc[NT], *bs[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int64_t m = m0 + 16 * i + r, row = m < p.M ? m : p.M - 1;
      ac[i] = p.a.codes + row * p.a.ldq;
      as[i] = p.a.scales + row * p.a.lds;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t n = n0 + 16 * j + r, row = n < p.N ? n : p.N - 1;
      bc[j] = p.b.codes + row * p.b.ldq;
      bs[j] = p.b.scales + row * p.b.lds;
    }
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave * U; s0 < steps; s0 += W * U) {
      i32x4 a[U][MT], b[U][NT];
      int sa[U][MT], sb[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int block = 4 * (s0 + u) + q;
        const bool live = block < nb;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          a[u][i] = live ? *reinterpret_cast<const i32x4*>(ac[i] + (int64_t)block * 16) : i32x4{0, 0, 0, 0};
          sa[u][i] = live ? as[i][block] : 127;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b[u][j] = live ? *reinterpret_cast<const i32x4*>(bc[j] + (int64_t)block * 16) : i32x4{0, 0, 0, 0};
          sb[u][j] = live ? bs[j][block] : 127;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = mfma_fp4(b[u][j], sb[u][j], a[u][i], sa[u][i], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4*>(&sums[wave][16 * i + r][16 * j + 4 * q]) = acc[i][j];
    __syncthreads();
    for (int e = threadIdx.x; e < BM * BN / 4; e += 64 * W) {
      const int m = e / (BN / 4), n = e % (BN / 4) * 4;
      f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][m][n]);
#pragma unroll
      for (int w = 1; w < W; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][m][n]);
      if (m0 + m < p.M && n0 + n < p.N) store4<DT>(p, m0 + m, n0 + n, v);
    }
    __syncthreads();
  }
}

template <int DT, int MT, int NT, int W, int U>
hipError_t launch_direct(const MatmulArgs& a, hipStream_t stream) {
  const int tiles_n = (a.N + 16 * NT - 1) / (16 * NT);
  const int64_t tiles = (int64_t)tiles_n * ((a.M + 16 * MT - 1) / (16 * MT));
  const int64_t most = 1 << 22;  // work-items of a grid: below 2^32
  hipLaunchKernelGGL((matmul_direct<DT, MT, NT, W, U>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(64 * W), 0,
                     stream, a, tiles_n, tiles);
  return hipGetLastError();
}

// The pipelined kernel: a workgroup of four waves computes BM x BN, each
// wave WM x WN in 16 x 16 blocks, 256 k (128 bytes a row) per slice through
// two LDS stages.
//  * Codes go from memory to LDS with 16-byte LDS-direct copies, chunk q of
//    row r at position q ^ (r/2)%8 of its 128-byte row, so that the 16 rows
//    of an operand read hit distinct banks.
//  * Scales: 8 bytes per row and slice, copied as two 4-byte pieces, read a
//    byte at a time straight into the instruction's scale operand (the four
//    lanes of a row read the same word).  In the last slice the blocks past
//    the matrix read zeros kept behind the scales instead, since a row's
//    bytes past its blocks may be anything (255 would be NaN).
//  * A k step is MB x NB matrix instructions in a fixed order; the next
//    step's operand reads and the copies of the slice after next are placed
//    between them.  One barrier per slice, before its last step (whose
//    operands are in registers by then).
// The operands are range-checked by the descriptors' and lanes' offsets:
// rows and blocks past the matrix load zeros.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  static constexpr int MB = WM / 16, NB = WN / 16, NMMA = MB * NB;
  static constexpr int ROW = 128, KB = 8;  // bytes and blocks per row and slice
  static constexpr int A_STAGE = BM * ROW, B_STAGE = BN * ROW;
  static constexpr int IA = A_STAGE / 1024 / NW, IB = B_STAGE / 1024 / NW;
  static constexpr int SA = BM * KB / 256 / NW, SB = BN * KB / 256 / NW;
  static constexpr int LPS = IA + IB + SA + SB;
  static_assert(IA > 0 && IB > 0 && SA > 0 && SB > 0, "copies split over the waves");
  __host__ __device__ static constexpr int byte(int r, int q) { return swz_off(r, q, ROW); }
  // Scales of fragment f: 16 rows on.
  static constexpr int SF = 16 * KB;
  static constexpr int SA_STAGE = BM * KB + MB * SF, SB_STAGE = BN * KB + NB * SF;
  // Slots among a step's NMMA instructions: operand f (A's, then B's), copy c.
  __host__ __device__ static constexpr int rd_slot(int f) { return f * NMMA / (MB + NB); }
  __host__ __device__ static constexpr int cp_slot(int c) { return c * NMMA / LPS; }
};

template <class S>
struct Copies {
  unsigned a[S::IA], b[S::IB], as[S::SA], bs[S::SB];
};

// Copy C of a slice, whose descriptors start at it; `left` blocks of the
// matrix are from its first on (<= 0: there is no such slice).
template <class S, int C>
__device__ __forceinline__ void copy_one(const uint8_t* Ab, const uint8_t* Bb, const uint8_t* As, const uint8_t* Bs,
                                         const Copies<S>& o, int64_t slice, int left, uint8_t* la,
                                         uint8_t* lb, uint8_t* lsa, uint8_t* lsb, int wave, int qa, int qb, int sw) {
  // (Device pass only: the host pass does not know the descriptor type.)
#if defined(__HIP_DEVICE_COMPILE__)
  const int range = left > 0 ? 0x7fffffff : 0;
  if constexpr (C < S::IA) {
    constexpr int i = C;
    const unsigned off = qa < left ? o.a[i] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(Ab + slice * S::ROW, range),
                                             (lds_void*)(la + 1024 * (i * S::NW + wave)), 16, off, 0, 0, 0);
  } else if constexpr (C < S::IA + S::IB) {
    constexpr int i = C - S::IA;
    const unsigned off = qb < left ? o.b[i] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(Bb + slice * S::ROW, range),
                                             (lds_void*)(lb + 1024 * (i * S::NW + wave)), 16, off, 0, 0, 0);
  } else if constexpr (C < S::IA + S::IB + S::SA) {
    constexpr int i = C - S::IA - S::IB;
    const unsigned off = sw < left ? o.as[i] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(As + slice * S::KB, range),
                                             (lds_void*)(lsa + 256 * (i * S::NW + wave)), 4, off, 0, 0, 0);
  } else {
    constexpr int i = C - S::IA - S::IB - S::SA;
    const unsigned off = sw < left ? o.bs[i] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(Bs + slice * S::KB, range),
                                             (lds_void*)(lsb + 256 * (i * S::NW + wave)), 4, off, 0, 0, 0);
  }
#endif
}

template <int DT, class S, bool EPI>
__global__ void __launch_bounds__(64 * S::NW)
matmul_pipe(MatmulArgs p, TileMap map, int vec) {
  constexpr int MB = S::MB, NB = S::NB;
  __shared__ __attribute__((aligned(1024))) uint8_t a0[S::A_STAGE], b0[S::B_STAGE], a1[S::A_STAGE], b1[S::B_STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[S::SA_STAGE], sb0[S::SB_STAGE], sa1[S::SA_STAGE], sb1[S::SB_STAGE];
  int tm, tn;
  tile_of_block(blockIdx.x, map, tm, tn);
  // (Said to be uniform: the descriptors have to be in scalar registers.)
  const int m0 = __builtin_amdgcn_readfirstlane(tm * S::BM), n0 = __builtin_amdgcn_readfirstlane(tn * S::BN);
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / S::WAVES_N) * S::WM, wn0 = (wave % S::WAVES_N) * S::WN;
  const int nb = (p.K + BLOCK - 1) / BLOCK;
  const int T = (nb + S::KB - 1) / S::KB;
  const uint8_t* Ab = p.a.codes + (int64_t)m0 * p.a.ldq;
  const uint8_t* Bb = p.b.codes + (int64_t)n0 * p.b.ldq;
  const uint8_t* As = p.a.scales + (int64_t)m0 * p.a.lds;
  const uint8_t* Bs = p.b.scales + (int64_t)n0 * p.b.lds;
  // This lane's place in the copies: 8 rows of 8 chunks, 32 rows of two
  // scale words; a chunk's index is the same for all copies of an operand.
  Copies<S> o;
  const int qa = (l % 8) ^ swz_row(8 * wave + l / 8, S::ROW), qb = qa;
  static_assert(S::NW % 2 == 0, "8 NW rows on, the chunk XOR repeats");
  const int sw = 4 * (l % 2);
#pragma unroll
  for (int i = 0; i < S::IA; ++i) {
    const int row = 8 * (i * S::NW + wave) + l / 8;
    o.a[i] = m0 + row < p.M ? (unsigned)(row * (int)p.a.ldq + 16 * qa) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::IB; ++i) {
    const int row = 8 * (i * S::NW + wave) + l / 8;
    o.b[i] = n0 + row < p.N ? (unsigned)(row * (int)p.b.ldq + 16 * qb) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::SA; ++i) {
    const int row = 32 * (i * S::NW + wave) + l / 2;
    o.as[i] = m0 + row < p.M ? (unsigned)(row * (int)p.a.lds + sw) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::SB; ++i) {
    const int row = 32 * (i * S::NW + wave) + l / 2;
    o.bs[i] = n0 + row < p.N ? (unsigned)(row * (int)p.b.lds + sw) : OOB;
  }
  for (int i = tid; i < MB * S::SF / 4; i += 64 * S::NW)
    reinterpret_cast<unsigned*>(sa0 + S::BM * S::KB)[i] = reinterpret_cast<unsigned*>(sa1 + S::BM * S::KB)[i] = 0u;
  for (int i = tid; i < NB * S::SF / 4; i += 64 * S::NW)
    reinterpret_cast<unsigned*>(sb0 + S::BN * S::KB)[i] = reinterpret_cast<unsigned*>(sb1 + S::BN * S::KB)[i] = 0u;
  // Operand reads: byte offsets of the two steps' first fragments.
  int a_fb[2], b_fb[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    a_fb[j] = S::byte(wm0 + r, 4 * j + q);
    b_fb[j] = S::byte(wn0 + r, 4 * j + q);
  }
  const int sa_fb = (wm0 + r) * S::KB + q, sb_fb = (wn0 + r) * S::KB + q;

  i32x4 fa[2][MB], fb[2][NB];
  int ga[2][MB], gb[2][NB];
  f32x4 acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#if defined(__HIP_DEVICE_COMPILE__)
      asm volatile("" : "+a"(acc[j][i]));
#endif
    }
  mfma_guard();

  // Operand f of step j of slice t into register set `buf`.
  auto read_op = [&](int buf, const uint8_t* la, const uint8_t* lb, const uint8_t* lsa, const uint8_t* lsb, int j, int t,
                     auto F) __attribute__((always_inline)) {
    constexpr int f = decltype(F)::value;
    const bool live = S::KB * t + 4 * j + q < nb;
    if constexpr (f < MB) {
      fa[buf][f] = *(const lds_i32x4*)(la + a_fb[j] + f * 16 * S::ROW);
      ga[buf][f] = *(const lds_u8*)(lsa + (live ? sa_fb + 4 * j : S::BM * S::KB) + f * S::SF);
    } else {
      constexpr int g = f - MB;
      fb[buf][g] = *(const lds_i32x4*)(lb + b_fb[j] + g * 16 * S::ROW);
      gb[buf][g] = *(const lds_u8*)(lsb + (live ? sb_fb + 4 * j : S::BN * S::KB) + g * S::SF);
    }
  };
  auto step = [&](int cur, auto&& rd, auto&& cp) __attribute__((always_inline)) {
    static_for([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      mfma_fp4_asm(acc[i / MB][i % MB], fb[cur][i / MB], fa[cur][i % MB], gb[cur][i / MB], ga[cur][i % MB]);
      static_for([&](auto F) __attribute__((always_inline)) {
        if constexpr (S::rd_slot(decltype(F)::value) == i) rd(F);
      }, std::make_integer_sequence<int, MB + NB>{});
      static_for([&](auto C) __attribute__((always_inline)) {
        if constexpr (S::cp_slot(decltype(C)::value) == i) cp(C);
      }, std::make_integer_sequence<int, S::LPS>{});
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, S::NMMA>{});
  };
  // Slice t from stage 0 or 1.
  auto slice = [&](int t, auto C_) __attribute__((always_inline)) {
    constexpr int c = decltype(C_)::value;
    uint8_t *la = c ? a1 : a0, *lb = c ? b1 : b0, *lsa = c ? sa1 : sa0, *lsb = c ? sb1 : sb0;
    uint8_t *na = c ? a0 : a1, *nbp = c ? b0 : b1, *nsa = c ? sa0 : sa1, *nsb = c ? sb0 : sb1;
    step(0, [&](auto F) __attribute__((always_inline)) { read_op(1, la, lb, lsa, lsb, 1, t, F); }, [](auto) {});
    loop_barrier();  // slice t + 1 landed, stage c read by every wave
    __builtin_amdgcn_sched_barrier(0);
    step(1, [&](auto F) __attribute__((always_inline)) { read_op(0, na, nbp, nsa, nsb, 0, t + 1, F); },
         [&](auto Q) __attribute__((always_inline)) {
           copy_one<S, decltype(Q)::value>(Ab, Bb, As, Bs, o, t + 2, nb - S::KB * (t + 2), la, lb, lsa, lsb, wave, qa,
                                           qb, sw);
         });
  };
  if (T > 0) {
    static_for([&](auto Q) __attribute__((always_inline)) {
      copy_one<S, decltype(Q)::value>(Ab, Bb, As, Bs, o, 0, nb, a0, b0, sa0, sb0, wave, qa, qb, sw);
    }, std::make_integer_sequence<int, S::LPS>{});
    static_for([&](auto Q) __attribute__((always_inline)) {
      copy_one<S, decltype(Q)::value>(Ab, Bb, As, Bs, o, 1, nb - S::KB, a1, b1, sa1, sb1, wave, qa, qb, sw);
    }, std::make_integer_sequence<int, S::LPS>{});
    loop_barrier();
    static_for([&](auto F) __attribute__((always_inline)) { read_op(0, a0, b0, sa0, sb0, 0, 0, F); },
               std::make_integer_sequence<int, MB + NB>{});
    int t = 0;
    for (; t + 2 <= T; t += 2) {
      slice(t, IC<0>{});
      slice(t + 1, IC<1>{});
    }
    mfma_guard();
    if (t < T) slice(t, IC<0>{});
    __builtin_amdgcn_s_waitcnt(0x0070);
  }
  mfma_guard();

  typedef typename TypeOf<DT>::type Out;
  const int rows = p.M - (m0 + wm0), cols = p.N - (n0 + wn0);
  const Out* C = static_cast<Out*>(p.C) + (int64_t)(m0 + wm0) * p.ldc + (n0 + wn0);
  auto store = [&](auto VEC) __attribute__((always_inline)) {
    f32x4 bias[NB];
    if constexpr (EPI) {
#pragma unroll
      for (int j = 0; j < NB; ++j) bias[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (p.epi.bias) load_block_row<GEMM_DTYPE_F32, NB, false>(p.epi.bias + n0 + wn0, 0u, cols, bias, q);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int m = 16 * i + r;
      const unsigned row = m < rows ? (unsigned)m * (unsigned)(p.ldc * (int)sizeof(Out)) : OOB;
      f32x4 v[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) v[j] = acc[j][i];
      if constexpr (EPI) {
        f32x4 old[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) old[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (p.epi.beta != 0.f) load_block_row<DT, NB, decltype(VEC)::value>(C, row, cols, old, q);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = epi_value(p.epi, v[j][e], old[j][e], bias[j][e]);
      }
      store_block_row<DT, NB, decltype(VEC)::value>(C, row, cols, v, q);
    }
  };
  if (vec) store(std::true_type{});
  else store(std::false_type{});
}

template <int DT, class S>
hipError_t launch_pipe(const MatmulArgs& a, hipStream_t stream) {
  TileMap map{(a.M + S::BM - 1) / S::BM, (a.N + S::BN - 1) / S::BN, GEMM_ORDER_XCD, 4, kXcds};
  const int es = DT == GEMM_DTYPE_F32 ? 4 : 2;
  const int vec = ((uintptr_t)a.C % 16 == 0 && a.ldc * es % 16 == 0 && a.N * es % 16 == 0) ? 1 : 0;
  const dim3 grid((unsigned)(map.tiles_m * map.tiles_n)), block(64 * S::NW);
  if (a.epi.on)
    hipLaunchKernelGGL((matmul_pipe<DT, S, true>), grid, block, 0, stream, a, map, vec);
  else
    hipLaunchKernelGGL((matmul_pipe<DT, S, false>), grid, block, 0, stream, a, map, vec);
  return hipGetLastError();
}

// What the pipelined kernel takes: scales in 4-byte words, a tile's rows
// within 31 bits, a grid below 2^32 work-items.
bool pipe_ok(const MatmulArgs& a) {
  const int64_t far = (int64_t)0x7fffffff / 256 - 4096;
  return a.K > 0 && (uintptr_t)a.a.scales % 4 == 0 && a.a.lds % 4 == 0 && (uintptr_t)a.b.scales % 4 == 0 &&
         a.b.lds % 4 == 0 && a.a.ldq < far && a.b.ldq < far && a.a.lds < far && a.b.lds < far && a.ldc < far / 4 &&
         (int64_t)((a.M + 127) / 128) * ((a.N + 127) / 128) < (1 << 23);
}

template <int DT>
hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 16) return launch_direct<DT, 1, 1, 8, 4>(a, stream);
  if (!pipe_ok(a)) return launch_direct<DT, 4, 4, 4, 1>(a, stream);
  // 256 x 256 tiles reuse each operand byte twice as often, 128 x 128 ones
  // fill the 256 CUs with a quarter of the outputs (4096^3: 39 against
  // 50 us; 2048^3: 19 against 10 us).
  const int64_t tiles = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  if (tiles >= 192) return launch_pipe<DT, Tile<256, 256, 128, 128>>(a, stream);
  return launch_pipe<DT, Tile<128, 128, 64, 64>>(a, stream);
}

}  // namespace

hipError_t launch_matmul(int c_dtype, const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  return c_dtype == GEMM_DTYPE_F32   ? launch<GEMM_DTYPE_F32>(a, stream)
         : c_dtype == GEMM_DTYPE_F16 ? launch<GEMM_DTYPE_F16>(a, stream)
                                     : launch<GEMM_DTYPE_BF16>(a, stream);
}

}  // namespace mx
}  // namespace gemm

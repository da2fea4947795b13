// The pipelined product of two E2M1 matrices (see mx_matmul.hip), one file
// for every combination of MX_DTYPE (type of C), MX_SIDE (tile) and MX_SC
// (scale pieces): compiled once for each.
#if !defined(MX_DTYPE) || !defined(MX_SIDE) || !defined(MX_SC)
#error "compiled once for every MX_DTYPE, MX_SIDE and MX_SC"
#endif

#include "mx_pipe.h"

namespace gemm {
namespace mx {
namespace {

// The pipelined kernel: a workgroup of four waves computes BM x BN, each
// wave WM x WN in 16 x 16 blocks, 256 k (128 bytes a row) per slice through
// two LDS stages.
//  * Codes go from memory to LDS with 16-byte LDS-direct copies.  A 16-byte
//    read serves 16 lanes at a time, rows 0-3 and 12-15 of an even lane group
//    with rows 4-11 of the next (or the other way round); with step j's chunk
//    of group q at position (4j + q) ^ (r/2)%8 of row r's 128 bytes, those
//    hit distinct banks (counted alone: no conflict cycle).
//  * Scales go to LDS for two slices at a time, 16 bytes of a row (SC = 16:
//    one copy a wave and operand; SC = 4, for scale rows that are only 4-byte
//    aligned, four).  A slice's two steps take blocks 2q and 2q + 1 for lane
//    group q, so that a lane's scales for both come with one read (of the
//    word that two groups share), and the instruction picks the byte.  A
//    bit-field extraction takes them out of the word and clears those past
//    the matrix' blocks, which may be anything (255 would be NaN).
//    (8192^3: 244 us; 273 us with 8 bytes a slice in 4-byte copies and a byte
//    read for each step.)  Those reads, of words 16 bytes apart, are the
//    loop's bank conflicts: 2 of each one's 4 LDS cycles, 17 % of all.
//  * A k step is MB x NB matrix instructions in a fixed order; the next
//    step's operand reads and the copies of the slice after next are placed
//    between them.  One barrier per slice, before its last step (whose
//    operands are in registers by then).
// The operands are range-checked by the lanes' offsets: rows and blocks past
// the matrix load zeros.
template <int BM_, int BN_, int WM_, int WN_, int SC_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, SC = SC_;
  static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  static constexpr int MB = WM / 16, NB = WN / 16, NMMA = MB * NB;
  static constexpr int ROW = 128, KB = 8;  // bytes and blocks per row and slice
  static constexpr int A_STAGE = BM * ROW, B_STAGE = BN * ROW;
  static constexpr int IA = A_STAGE / 1024 / NW, IB = B_STAGE / 1024 / NW;
  // Scale copies of a wave, for two slices: rows of 16 bytes.
  static constexpr int SROW = 16, SPI = 64 * SC / SROW;  // rows of one copy
  __host__ __device__ static constexpr int scale_copies(int rows) { return (rows + SPI * NW - 1) / (SPI * NW); }
  static constexpr int SA = scale_copies(BM), SB = scale_copies(BN);
  static constexpr int SA_STAGE = SA * SPI * NW * SROW, SB_STAGE = SB * SPI * NW * SROW;
  static_assert(IA > 0 && IB > 0 && NW % 2 == 0, "copies split over the waves; 8 NW rows on, the chunk XOR repeats");
  static_assert(SC == 4 || SC == 16, "scale pieces");
  // Position `slot` of a row, XORed by the row; the chunk that belongs there.
  __host__ __device__ static constexpr int byte(int r, int slot) { return swz_off(r, slot, ROW); }
  __host__ __device__ static constexpr int chunk_at(int slot) { return 2 * (slot % 4) + slot / 4; }
  // Slots among a step's NMMA instructions: operand f (A's, then B's); its
  // scales and their extraction, at least 6 instructions later and as many
  // before the next step; copy c of n.
  static constexpr int F = MB + NB;
  struct Read {
    __host__ __device__ static constexpr int at(int f) { return f * NMMA / F; }
  };
  struct Scale {
    __host__ __device__ static constexpr int at(int f) { return f * NMMA / (2 * F); }
  };
  struct Take {
    __host__ __device__ static constexpr int at(int f) { return Scale::at(f) + 3 * NMMA / 8; }
  };
  template <int N>
  struct Copy {
    __host__ __device__ static constexpr int at(int c) { return c * NMMA / N; }
  };
};

// A lane's offsets in the copies of a slice (codes) and of two (scales).
template <class S>
struct Copies {
  unsigned a[S::IA], b[S::IB], as[S::SA], bs[S::SB];
  int q, sw;  // its chunk of a row; its first scale block of 16
};

// Copy C of a slice's codes (A's, then B's), whose descriptors start at it;
// `left` blocks of the matrix are from its first on (<= 0: no such slice).
template <class S, int C>
__device__ __forceinline__ void copy_codes(const uint8_t* A, const uint8_t* B, const Copies<S>& o, int64_t slice, int left,
                                           uint8_t* la, uint8_t* lb, int wave) {
  // (Device pass only: the host pass does not know the descriptor type.)
#if defined(__HIP_DEVICE_COMPILE__)
  const int range = left > 0 ? 0x7fffffff : 0;
  if constexpr (C < S::IA) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(A + slice * S::ROW, range),
                                             (lds_void*)(la + 1024 * (C * S::NW + wave)), 16, o.q < left ? o.a[C] : OOB, 0,
                                             0, 0);
  } else {
    constexpr int i = C - S::IA;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(B + slice * S::ROW, range),
                                             (lds_void*)(lb + 1024 * (i * S::NW + wave)), 16, o.q < left ? o.b[i] : OOB, 0,
                                             0, 0);
  }
#endif
}

// The same of the scales of a pair of slices.
template <class S, int C>
__device__ __forceinline__ void copy_scales(const uint8_t* A, const uint8_t* B, const Copies<S>& o, int64_t pair, int left,
                                            uint8_t* la, uint8_t* lb, int wave) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int range = left > 0 ? 0x7fffffff : 0;
  constexpr int BYTES = S::SPI * S::SROW;  // of one copy
  if constexpr (C < S::SA) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(A + pair * S::SROW, range),
                                             (lds_void*)(la + BYTES * (C * S::NW + wave)), S::SC,
                                             o.sw < left ? o.as[C] : OOB, 0, 0, 0);
  } else {
    constexpr int i = C - S::SA;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(B + pair * S::SROW, range),
                                             (lds_void*)(lb + BYTES * (i * S::NW + wave)), S::SC,
                                             o.sw < left ? o.bs[i] : OOB, 0, 0, 0);
  }
#endif
}

template <int DT, class S, bool EPI>
__global__ void __launch_bounds__(64 * S::NW)
matmul_pipe(MatmulArgs p, TileMap map, int vec) {
  constexpr int MB = S::MB, NB = S::NB, F = S::F, NC = S::IA + S::IB, NSC = S::SA + S::SB;
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
  // A code copy is 8 rows of 8 chunks, the chunk index the same for all of a
  // wave's; a scale copy SPI rows of 16 bytes.
  Copies<S> o;
  o.q = S::chunk_at((l % 8) ^ swz_row(8 * wave + l / 8, S::ROW));
  o.sw = S::SC == 4 ? 4 * (l % 4) : 0;
#pragma unroll
  for (int i = 0; i < S::IA; ++i) {
    const int row = 8 * (i * S::NW + wave) + l / 8;
    o.a[i] = m0 + row < p.M ? (unsigned)(row * (int)p.a.ldq + 16 * o.q) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::IB; ++i) {
    const int row = 8 * (i * S::NW + wave) + l / 8;
    o.b[i] = n0 + row < p.N ? (unsigned)(row * (int)p.b.ldq + 16 * o.q) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::SA; ++i) {
    const int row = S::SPI * (i * S::NW + wave) + l / (S::SROW / S::SC);
    o.as[i] = row < S::BM && m0 + row < p.M ? (unsigned)(row * (int)p.a.lds + o.sw) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::SB; ++i) {
    const int row = S::SPI * (i * S::NW + wave) + l / (S::SROW / S::SC);
    o.bs[i] = row < S::BN && n0 + row < p.N ? (unsigned)(row * (int)p.b.lds + o.sw) : OOB;
  }
  // Operand reads: byte offsets of the two steps' first fragments.
  int a_fb[2], b_fb[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    a_fb[j] = S::byte(wm0 + r, 4 * j + q);
    b_fb[j] = S::byte(wn0 + r, 4 * j + q);
  }
  const int sa_fb = (wm0 + r) * S::SROW + q / 2 * 4, sb_fb = (wn0 + r) * S::SROW + q / 2 * 4;

  i32x4 fa[2][MB], fb[2][NB];  // by step
  int ga[2][MB], gb[2][NB];    // by slice
  f32x4 acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  pin(acc);
  mfma_guard();

  // Operand f of step j from a stage.
  auto read_op = [&](const uint8_t* la, const uint8_t* lb, auto J, auto F_) __attribute__((always_inline)) {
    constexpr int j = decltype(J)::value, f = decltype(F_)::value;
    if constexpr (f < MB)
      fa[j][f] = *(const lds_i32x4*)(la + a_fb[j] + f * 16 * S::ROW);
    else
      fb[j][f - MB] = *(const lds_i32x4*)(lb + b_fb[j] + (f - MB) * 16 * S::ROW);
  };
  // Its scales in slice c of a pair, and their extraction: `bits` of them
  // belong to blocks inside the matrix.
  auto read_scale = [&](const uint8_t* lsa, const uint8_t* lsb, auto C_, auto F_) __attribute__((always_inline)) {
    constexpr int c = decltype(C_)::value, f = decltype(F_)::value;
    if constexpr (f < MB)
      ga[c][f] = (int)*(const lds_u32*)(lsa + sa_fb + 8 * c + f * 16 * S::SROW);
    else
      gb[c][f - MB] = (int)*(const lds_u32*)(lsb + sb_fb + 8 * c + (f - MB) * 16 * S::SROW);
  };
  const int from = 16 * (q % 2);
  auto take_scale = [&](int bits, auto C_, auto F_) __attribute__((always_inline)) {
    constexpr int c = decltype(C_)::value, f = decltype(F_)::value;
    if constexpr (f < MB)
      ga[c][f] = (int)__builtin_amdgcn_ubfe((unsigned)ga[c][f], from, bits);
    else
      gb[c][f - MB] = (int)__builtin_amdgcn_ubfe((unsigned)gb[c][f - MB], from, bits);
  };
  auto bits_of = [&](int t) __attribute__((always_inline)) {
    const int first = S::KB * t + 2 * q;
    return first + 1 < nb ? 16 : first < nb ? 8 : 0;
  };
  // Step j of a slice c; `between` runs after each instruction.
  auto step = [&](auto J, auto C_, auto&& between) __attribute__((always_inline)) {
    static_for([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value, j = decltype(J)::value, c = decltype(C_)::value;
      mfma_fp4_asm<j>(acc[i / MB][i % MB], fb[j][i / MB], fa[j][i % MB], gb[c][i / MB], ga[c][i % MB]);
      between(I);
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, S::NMMA>{});
  };
  auto at_slot = [&](auto I, auto SLOT, auto N, auto&& f) __attribute__((always_inline)) {
    static_for([&](auto X) __attribute__((always_inline)) {
      if constexpr (decltype(SLOT)::at(decltype(X)::value) == decltype(I)::value) f(X);
    }, std::make_integer_sequence<int, decltype(N)::value>{});
  };
  // Slice t: number c of its pair, whose scales are in buffer PAR.
  auto slice = [&](int t, auto C_, auto PAR) __attribute__((always_inline)) {
    constexpr int c = decltype(C_)::value, par = decltype(PAR)::value;
    uint8_t *la = c ? a1 : a0, *lb = c ? b1 : b0, *na = c ? a0 : a1, *nbp = c ? b0 : b1;
    // The next slice's scales: this pair's, or the next one's.
    constexpr int np = c ? 1 - par : par;
    uint8_t *nsa = np ? sa1 : sa0, *nsb = np ? sb1 : sb0;
    uint8_t *psa = par ? sa0 : sa1, *psb = par ? sb0 : sb1;  // the next pair's
    step(IC<0>{}, IC<c>{}, [&](auto I) __attribute__((always_inline)) {
      at_slot(I, typename S::Read{}, IC<F>{},
              [&](auto X) __attribute__((always_inline)) { read_op(la, lb, IC<1>{}, X); });
    });
    loop_barrier();  // slice t + 1 landed, stage c read by every wave
    __builtin_amdgcn_sched_barrier(0);
    const int bits = bits_of(t + 1);
    constexpr int n = c ? NC : NC + NSC;
    step(IC<1>{}, IC<c>{}, [&](auto I) __attribute__((always_inline)) {
      at_slot(I, typename S::Scale{}, IC<F>{},
              [&](auto X) __attribute__((always_inline)) { read_scale(nsa, nsb, IC<1 - c>{}, X); });
      at_slot(I, typename S::Read{}, IC<F>{},
              [&](auto X) __attribute__((always_inline)) { read_op(na, nbp, IC<0>{}, X); });
      at_slot(I, typename S::Take{}, IC<F>{},
              [&](auto X) __attribute__((always_inline)) { take_scale(bits, IC<1 - c>{}, X); });
      at_slot(I, typename S::template Copy<n>{}, IC<n>{}, [&](auto X) __attribute__((always_inline)) {
        constexpr int x = decltype(X)::value;
        if constexpr (x < NC)
          copy_codes<S, x>(Ab, Bb, o, t + 2, nb - S::KB * (t + 2), la, lb, wave);
        else
          copy_scales<S, x - NC>(As, Bs, o, t / 2 + 1, nb - S::KB * (t + 2), psa, psb, wave);
      });
    });
  };
  auto copy_slice = [&](int t, uint8_t* la, uint8_t* lb) __attribute__((always_inline)) {
    static_for([&](auto X) __attribute__((always_inline)) {
      copy_codes<S, decltype(X)::value>(Ab, Bb, o, t, nb - S::KB * t, la, lb, wave);
    }, std::make_integer_sequence<int, NC>{});
  };
  if (T > 0) {
    copy_slice(0, a0, b0);
    static_for([&](auto X) __attribute__((always_inline)) {
      copy_scales<S, decltype(X)::value>(As, Bs, o, 0, nb, sa0, sb0, wave);
    }, std::make_integer_sequence<int, NSC>{});
    copy_slice(1, a1, b1);
    loop_barrier();
    static_for([&](auto X) __attribute__((always_inline)) {
      read_op(a0, b0, IC<0>{}, X);
      read_scale(sa0, sb0, IC<0>{}, X);
    }, std::make_integer_sequence<int, F>{});
    static_for([&](auto X) __attribute__((always_inline)) { take_scale(bits_of(0), IC<0>{}, X); },
               std::make_integer_sequence<int, F>{});
    mfma_guard();
    int t = 0;
    for (; t + 4 <= T; t += 4) {
      slice(t, IC<0>{}, IC<0>{});
      slice(t + 1, IC<1>{}, IC<0>{});
      slice(t + 2, IC<0>{}, IC<1>{});
      slice(t + 3, IC<1>{}, IC<1>{});
    }
    mfma_guard();
    if (t < T) {
      slice(t, IC<0>{}, IC<0>{});
      mfma_guard();
    }
    if (t + 1 < T) {
      slice(t + 1, IC<1>{}, IC<0>{});
      mfma_guard();
    }
    if (t + 2 < T) slice(t + 2, IC<0>{}, IC<1>{});
    __builtin_amdgcn_s_waitcnt(0x0070);
  }
  mfma_guard();
  pin(acc);  // (read after the guard only)

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

}  // namespace

template <int DT, int SIDE, int SC>
hipError_t launch_matmul_pipe(const MatmulArgs& a, hipStream_t stream) {
  typedef Tile<SIDE, SIDE, SIDE / 2, SIDE / 2, SC> S;
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

template hipError_t launch_matmul_pipe<MX_DTYPE, MX_SIDE, MX_SC>(const MatmulArgs&, hipStream_t);

}  // namespace mx
}  // namespace gemm

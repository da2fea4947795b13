// The pipelined kernel of the weight gradient (see mx_wgrad.hip), one file
// for every combination of MX_DTYPE (type of dW or of the partial sums) and
// MX_SIDE (tile): compiled once for each.
#if !defined(MX_DTYPE) || !defined(MX_SIDE)
#error "compiled once for every MX_DTYPE and MX_SIDE"
#endif

#include "mx_pipe.h"

namespace gemm {
namespace mx {
namespace {

// The pipelined kernel: a workgroup of four waves computes BM features x BN
// columns, each wave WM x WN in 16 x 16 blocks, 64 tokens per slice through
// two LDS stages.
//  * The codes (token-contiguous, 64 bytes a feature and slice) and dY's
//    rows (as in memory) go to LDS with 16-byte LDS-direct copies; the codes
//    stay 8 bits wide there and are decoded on the way into the operand
//    registers, four conversions an operand, which run beside the matrix
//    core.  Lane group q takes tokens 16q + 8j .. + 7 of a slice in step j
//    (any order common to both operands will do), so that a feature's codes
//    for both steps are one 16-byte read and their scale, of block q/2, one
//    byte.  (8192 tokens, 4096 x 4096: 204 us; 214 us with 8 bytes a step,
//    tokens 32j + 8q, whose reads took 6 LDS cycles each, 4 of them in bank
//    conflicts.)
//  * dY's operands want token-contiguous values of a column: the transpose
//    read ds_read_b64_tr_b16 (in each group of 16 lanes, lane j gets element
//    j%4 of the 8-byte pieces that lanes j/4 + 4t point at).  Its rows'
//    16-byte chunks are XORed by 4(k%4) + (k/16)%2: step j's rows are 8j
//    further, which must not change the XOR.  2 of each transpose read's 4
//    LDS cycles are still bank conflicts, 36 % of the kernel's LDS cycles;
//    the codes' and scales' reads have none.
//  * Scales: one 4-byte word a feature (four blocks) with every slice;
//    blocks past the tokens read zeros kept behind them.
//  * The terms of dY are further tokens: the slices run over the tokens of
//    term 0, then term 1, and so on, with the same codes.
//  * A step (32 tokens: one block) is MB x NB matrix instructions in a
//    fixed order, with the next step's reads, its decoding and the copies of
//    the slice after next between them; one barrier per slice, before its
//    last step.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = 64;
  static constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
  static constexpr int MB = WM / 16, NB = WN / 16, NMMA = MB * NB;
  static constexpr int A_ROW = BK, B_ROW = 2 * BN;
  static constexpr int A_STAGE = BM * A_ROW, B_STAGE = BK * B_ROW;
  static constexpr int IA = A_STAGE / 1024 / NW, IB = B_STAGE / 1024 / NW;
  static constexpr int LPS = IA + IB + 1;
  static constexpr int SF = 64;  // scale bytes of one fragment's 16 rows
  // One scale copy a wave; those past the features write zeros, behind the
  // scales, where zeros are wanted.
  static constexpr int S_STAGE = BM * 4 + MB * SF > 256 * NW ? BM * 4 + MB * SF : 256 * NW;
  static_assert(IA > 0 && IB > 0 && BM <= 64 * NW && B_ROW >= 256, "copies split over the waves");
  __host__ __device__ static constexpr int b_swz(int k) { return (4 * (k % 4)) ^ ((k / 16) % 2); }
  __host__ __device__ static constexpr int b_byte(int k, int n) {
    return k * B_ROW + 16 * ((n / 8) ^ b_swz(k)) + 2 * (n % 8);
  }
  // Chunk q of feature row r: 16-byte reads serve rows 0-3 and 12-15 of one
  // lane group with rows 4-11 of its neighbour, which this XOR (0, 3, 2, 1
  // by fours of rows) sends to distinct banks.
  __host__ __device__ static constexpr int a_swz(int r) { return (4 - r / 4 % 4) % 4; }
  __host__ __device__ static constexpr int a_byte(int r, int q) { return r * A_ROW + 16 * (q ^ a_swz(r)); }
  // Slots among a step's NMMA instructions.
  __host__ __device__ static constexpr int a_slot(int f) { return f * NMMA / (4 * MB); }
  __host__ __device__ static constexpr int b_slot(int g) { return NMMA / 4 + g * NMMA / (2 * NB); }
  __host__ __device__ static constexpr int dec_slot(int f) { return 3 * NMMA / 8 + f * NMMA / (2 * MB); }
  __host__ __device__ static constexpr int cp_slot(int c) { return c * NMMA / LPS; }
};

template <class S>
struct Copies {
  unsigned a[S::IA], b[S::IB], s;
};

// Copy C of a slice: the codes of `ka` bytes, rows of dY `yb` bytes and the
// scales `ks` bytes into their operands, with `a_left` code bytes a row and
// `y_left` bytes of dY from there on (0: no such slice).
template <class S, int C>
__device__ __forceinline__ void copy_one(const uint8_t* A, const uint8_t* Y, const uint8_t* Sc, const Copies<S>& o,
                                         int64_t ka, int64_t yb, int64_t ks, int a_left, int y_left, uint8_t* la,
                                         uint8_t* lb, uint8_t* ls, int wave, int qa) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int range = a_left > 0 ? 0x7fffffff : 0;
  if constexpr (C < S::IA) {
    const unsigned off = 16 * qa < a_left ? o.a[C] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(A + ka, range), (lds_void*)(la + 1024 * (C * S::NW + wave)), 16,
                                             off, 0, 0, 0);
  } else if constexpr (C < S::IA + S::IB) {
    constexpr int i = C - S::IA;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(Y + yb, y_left), (lds_void*)(lb + 1024 * (i * S::NW + wave)), 16,
                                             o.b[i], 0, 0, 0);
  } else {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(Sc + ks, range), (lds_void*)(ls + 256 * wave), 4, o.s, 0, 0, 0);
  }
#endif
}

template <int DT, class S, bool EPI>
__global__ void __launch_bounds__(64 * S::NW)
wgrad_pipe(WgradPipeArgs p, TileMap map, int vec) {
  constexpr int MB = S::MB, NB = S::NB;
  __shared__ __attribute__((aligned(1024))) uint8_t a0[S::A_STAGE], b0[S::B_STAGE], a1[S::A_STAGE], b1[S::B_STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t s0[S::S_STAGE], s1[S::S_STAGE];
  int tm, tn;
  tile_of_block(blockIdx.x, map, tm, tn);
  // (Said to be uniform: the descriptors have to be in scalar registers.)
  const int m0 = __builtin_amdgcn_readfirstlane(tm * S::BM), n0 = __builtin_amdgcn_readfirstlane(tn * S::BN);
  const int tid = threadIdx.x, l = tid & 63, r = l % 16, q = l / 16;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm0 = (wave / S::WAVES_N) * S::WM, wn0 = (wave % S::WAVES_N) * S::WN;
  // This workgroup's tokens: [t0, t1), pairs of slices of 128 of them, per
  // term; its code bytes end at whole blocks.
  const int64_t t0 = (int64_t)blockIdx.y * p.chunk;
  const int t1 = (int)(t0 + p.chunk < p.T ? t0 + p.chunk : p.T);
  const int len = t1 - (int)t0;
  const int bytes = (len + BLOCK - 1) / BLOCK * BLOCK;
  const int pairs = (len + 2 * S::BK - 1) / (2 * S::BK), P = pairs * p.terms;
  const uint8_t* A = p.x.codes + (int64_t)m0 * p.x.ldq + t0;
  const uint8_t* Sc = p.x.scales + (int64_t)m0 * p.x.lds + t0 / BLOCK;
  const uint8_t* Y = reinterpret_cast<const uint8_t*>(p.y + t0 * p.ldy + n0);
  const int y_row = 2 * (int)p.ldy;
  const int64_t y_plane = 2 * p.plane;
  const int y_cols = 2 * ((p.N + 7) / 8 * 8 - n0);  // bytes of a row from here on
  // dY's bytes from a slice on that has `left` tokens.
  auto y_range = [&](int left) __attribute__((always_inline)) {
    const int rows = left < S::BK ? left : S::BK, n = (rows - 1) * y_row + y_cols;
    return rows > 0 ? n : 0;
  };

  Copies<S> o;
  const int qa = (l % 4) ^ S::a_swz(l / 4);
#pragma unroll
  for (int i = 0; i < S::IA; ++i) {
    const int row = 16 * (i * S::NW + wave) + l / 4;
    o.a[i] = m0 + row < p.F ? (unsigned)(row * (int)p.x.ldq + 16 * qa) : OOB;
  }
#pragma unroll
  for (int i = 0; i < S::IB; ++i) {
    const int at = 1024 * (i * S::NW + wave) + 16 * l;
    const int k = at / S::B_ROW, c = (at % S::B_ROW / 16) ^ S::b_swz(k);
    o.b[i] = n0 + 8 * c < p.N ? (unsigned)(k * y_row + 16 * c) : OOB;  // (rows past the tokens: out of range)
  }
  {
    const int row = 64 * wave + l;
    o.s = row < S::BM && m0 + row < p.F ? (unsigned)(row * (int)p.x.lds) : OOB;
  }
  for (int i = tid; i < MB * S::SF / 4; i += 64 * S::NW)
    reinterpret_cast<unsigned*>(s0 + S::BM * 4)[i] = reinterpret_cast<unsigned*>(s1 + S::BM * 4)[i] = 0u;
  const int a_fb = S::a_byte(wm0 + r, q);
  int b_fb[NB];
#pragma unroll
  for (int g = 0; g < NB; ++g) b_fb[g] = S::b_byte(16 * q + r / 4, wn0 + 16 * g + 4 * (r % 4));
  const int s_fb = (wm0 + r) * 4 + q / 2;

  i32x4 fa[2][MB], fb[2][NB];
  u32x4 raw[MB];  // a slice's codes and scales
  unsigned sc[MB];
  f32x4 acc[NB][MB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  pin(acc);
  mfma_guard();

  // Codes and scales of a slice whose block 0 is `block` of the workgroup's,
  // its scales the bytes 2c .. of their words.
  auto read_a = [&](const uint8_t* la, const uint8_t* ls, int c, int block, auto F) __attribute__((always_inline)) {
    constexpr int f = decltype(F)::value;
    raw[f] = __builtin_bit_cast(u32x4, *(const lds_i32x4*)(la + a_fb + f * 16 * S::A_ROW));
    sc[f] = *(const lds_u8*)(ls + (BLOCK * (block + q / 2) < bytes ? s_fb + 2 * c : S::BM * 4) + f * S::SF);
  };
  auto read_b = [&](int buf, const uint8_t* lb, int j, auto G) __attribute__((always_inline)) {
    constexpr int g = decltype(G)::value;
    const uint8_t* b = lb + b_fb[g] + 8 * j * S::B_ROW;
    const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)b));
    const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(b + 4 * S::B_ROW)));
    fb[buf][g] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
  };
  // Step j's operand f.
  auto decode = [&](int j, auto F) __attribute__((always_inline)) {
    constexpr int f = decltype(F)::value;
    const u32x2 w = {j ? raw[f][2] : raw[f][0], j ? raw[f][3] : raw[f][1]};
    fa[j][f] = __builtin_bit_cast(i32x4, decode8(w, scale_float(sc[f])));
  };
  auto step = [&](int cur, auto&& ra, auto&& rb, auto&& cp) __attribute__((always_inline)) {
    static_for([&](auto I) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value;
      mfma_bf16_asm(acc[i / MB][i % MB], fb[cur][i / MB], fa[cur][i % MB]);
      static_for([&](auto F) __attribute__((always_inline)) {
        if constexpr (S::a_slot(decltype(F)::value) == i) ra(F);
        if constexpr (S::dec_slot(decltype(F)::value) == i) decode(cur ^ 1, F);
      }, std::make_integer_sequence<int, MB>{});
      static_for([&](auto G) __attribute__((always_inline)) {
        if constexpr (S::b_slot(decltype(G)::value) == i) rb(G);
      }, std::make_integer_sequence<int, NB>{});
      static_for([&](auto C) __attribute__((always_inline)) {
        if constexpr (S::cp_slot(decltype(C)::value) == i) cp(C);
      }, std::make_integer_sequence<int, S::LPS>{});
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, S::NMMA>{});
  };
  // Slice c of pair pt (in its term) from stage c; the next pair is pair
  // ptn of term tnx (live: there is one).
  auto slice = [&](auto C_, int pt, int ptn, int tnx, bool live) __attribute__((always_inline)) {
    constexpr int c = decltype(C_)::value;
    uint8_t *la = c ? a1 : a0, *lb = c ? b1 : b0, *ls = c ? s1 : s0;
    uint8_t *na = c ? a0 : a1, *nbp = c ? b0 : b1, *ns = c ? s0 : s1;
    step(0, [](auto) {}, [&](auto G) __attribute__((always_inline)) { read_b(1, lb, 1, G); }, [](auto) {});
    loop_barrier();  // the next slice landed, stage c read by every wave
    __builtin_amdgcn_sched_barrier(0);
    const int k = 2 * S::BK * ptn + S::BK * c;
    const int left = (live ? len : 0) - k;
    step(1, [&](auto F) __attribute__((always_inline)) { read_a(na, ns, c ^ 1, c ? 4 * ptn : 4 * pt + 2, F); },
         [&](auto G) __attribute__((always_inline)) { read_b(0, nbp, 0, G); },
         [&](auto Q) __attribute__((always_inline)) {
           copy_one<S, decltype(Q)::value>(A, Y, Sc, o, k, tnx * y_plane + k * (int64_t)y_row, 4 * ptn, (live ? bytes : 0) - k,
                                           y_range(left), la, lb, ls, wave, qa);
         });
  };
  if (P > 0) {
    static_for([&](auto Q) __attribute__((always_inline)) {
      copy_one<S, decltype(Q)::value>(A, Y, Sc, o, 0, 0, 0, bytes, y_range(len), a0, b0, s0,
                                      wave, qa);
      copy_one<S, decltype(Q)::value>(A, Y, Sc, o, S::BK, S::BK * (int64_t)y_row, 0, bytes - S::BK,
                                      y_range(len - S::BK), a1, b1, s1, wave, qa);
    }, std::make_integer_sequence<int, S::LPS>{});
    loop_barrier();
    static_for([&](auto F) __attribute__((always_inline)) { read_a(a0, s0, 0, 0, F); },
               std::make_integer_sequence<int, MB>{});
    static_for([&](auto G) __attribute__((always_inline)) { read_b(0, b0, 0, G); }, std::make_integer_sequence<int, NB>{});
    static_for([&](auto F) __attribute__((always_inline)) { decode(0, F); }, std::make_integer_sequence<int, MB>{});
    mfma_guard();
    int pt = 0, term = 0;
    for (int i = 0; i < P; ++i) {
      int ptn = pt + 1, tnx = term;
      if (ptn == pairs) {
        ptn = 0;
        ++tnx;
      }
      const bool live = i + 1 < P;
      slice(IC<0>{}, pt, ptn, tnx, live);
      slice(IC<1>{}, pt, ptn, tnx, live);
      pt = ptn;
      term = tnx;
    }
    __builtin_amdgcn_s_waitcnt(0x0070);
  }
  mfma_guard();
  pin(acc);  // (read after the guard only)

  typedef typename TypeOf<DT>::type Out;
  const int rows = p.F - (m0 + wm0), cols = p.N - (n0 + wn0);
  const Out* C = static_cast<Out*>(p.C) + blockIdx.y * p.c_stride + (int64_t)(m0 + wm0) * p.ldc + (n0 + wn0);
  auto store = [&](auto VEC) __attribute__((always_inline)) {
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
        if (p.beta != 0.f) load_block_row<DT, NB, decltype(VEC)::value>(C, row, cols, old, q);
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[j][e] *= p.alpha;
            if (p.beta != 0.f) v[j][e] = __builtin_fmaf(p.beta, old[j][e], v[j][e]);
          }
      }
      store_block_row<DT, NB, decltype(VEC)::value>(C, row, cols, v, q);
    }
  };
  if (vec) store(std::true_type{});
  else store(std::false_type{});
}

}  // namespace

template <int CT, int SIDE>
hipError_t launch_wgrad_pipe(const WgradPipeArgs& a, int splits, hipStream_t stream) {
  typedef Tile<SIDE, SIDE, SIDE / 2, SIDE / 2> S;
  TileMap map{(a.F + S::BM - 1) / S::BM, (a.N + S::BN - 1) / S::BN, GEMM_ORDER_XCD, 4, kXcds};
  const int es = CT == GEMM_DTYPE_F32 ? 4 : 2;
  const int vec = ((uintptr_t)a.C % 16 == 0 && a.ldc * es % 16 == 0 && a.N * es % 16 == 0) ? 1 : 0;
  const dim3 grid((unsigned)(map.tiles_m * map.tiles_n), (unsigned)splits), block(64 * S::NW);
  if (a.alpha != 1.f || a.beta != 0.f)
    hipLaunchKernelGGL((wgrad_pipe<CT, S, true>), grid, block, 0, stream, a, map, vec);
  else
    hipLaunchKernelGGL((wgrad_pipe<CT, S, false>), grid, block, 0, stream, a, map, vec);
  return hipGetLastError();
}

template hipError_t launch_wgrad_pipe<MX_DTYPE, MX_SIDE>(const WgradPipeArgs&, int, hipStream_t);

}  // namespace mx
}  // namespace gemm

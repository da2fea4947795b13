// Weight gradient from an 8-bit activation checkpoint, dW = alpha X^T dY +
// beta dW (include/gemm_mx.h): a product summed over tokens, of the E4M3
// codes of X^T (F x T, blocks of 32 tokens) with dY (T x N, row-major).
//
// The bfloat16 matrix instruction takes both operands exactly.  A code is
// four significant bits times a power of two, so v_cvt_scalef32_pk_bf16_fp8
// (code and factor in, bfloat16 out) rounds nothing above bfloat16's
// subnormals.  A binary16 dY is the sum of two bfloat16 terms (8 + 3
// significant bits), an FP32 one of three (8 + 8 + 8), each a truncation of
// what the terms before it left, so the differences are exact; every term
// is one more matrix instruction on the same codes.
#include "mx_pipe.h"

namespace gemm {
namespace mx {
namespace {

// Eight codes (tokens in order) of one block -> eight bfloat16 values.
__device__ __forceinline__ u32x4 decode8(u32x2 w, float factor) {
  u32x4 v;
  v[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], factor, false));
  v[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], factor, true));
  v[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], factor, false));
  v[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], factor, true));
  return v;
}

// bfloat16 terms of a value of type YT.
template <int YT>
constexpr int kTerms = YT == GEMM_DTYPE_BF16 ? 1 : YT == GEMM_DTYPE_F16 ? 2 : 3;

// The terms' bit patterns, largest first.  Infinities and NaN: the first
// term alone (rounded, which keeps a NaN a NaN).
template <int YT>
__device__ __forceinline__ void split_terms(float x, unsigned short (&t)[kTerms<YT>]) {
  if constexpr (YT == GEMM_DTYPE_BF16) {
    t[0] = (unsigned short)(__builtin_bit_cast(unsigned, x) >> 16);
  } else {
    const unsigned bits = __builtin_bit_cast(unsigned, x);
    const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
    float left = x;
#pragma unroll
    for (int k = 0; k < kTerms<YT>; ++k) {
      const unsigned top = __builtin_bit_cast(unsigned, left) & 0xffff0000u;
      t[k] = (unsigned short)(top >> 16);
      left -= __builtin_bit_cast(float, top);
    }
    if (!finite) {
      t[0] = round16<true>(x);
#pragma unroll
      for (int k = 1; k < kTerms<YT>; ++k) t[k] = 0;
    }
  }
}

template <int DT>
__device__ __forceinline__ float read_as_float(const void* p, int64_t i) {
  return (float)static_cast<const typename TypeOf<DT>::type*>(p)[i];
}

// dW[f][n .. n+3] from its sums.
template <int DT>
__device__ __forceinline__ void store4(const WgradArgs& p, int64_t f, int64_t n, f32x4 acc) {
  typedef typename TypeOf<DT>::type T;
  typedef T t4 __attribute__((ext_vector_type(4)));
  T* c = static_cast<T*>(p.dW) + f * p.ldw + n;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[i] *= p.alpha;
    if (p.beta != 0.f && n + i < p.N) acc[i] = __builtin_fmaf(p.beta, (float)c[i], acc[i]);
  }
  if (n + 4 <= p.N && ((uintptr_t)c & (sizeof(t4) - 1)) == 0) {
    *reinterpret_cast<t4*>(c) = t4{(T)acc[0], (T)acc[1], (T)acc[2], (T)acc[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) c[i] = (T)acc[i];
  }
}

// The general kernel: any alignment of dY, every type.  A workgroup of four
// waves computes 64 features x 64 columns, 32 tokens (one block of the
// codes) at a time through LDS: the codes' values token-contiguous, dY's
// terms transposed to token-contiguous while they are staged.
template <int YT, int CT>
__global__ void __launch_bounds__(256)
wgrad_general(WgradArgs p, int tiles_n, int64_t tiles) {
  constexpr int NT = kTerms<YT>;
  constexpr int LD = 40;  // 32 tokens and padding: 80-byte rows spread the banks
  __shared__ __attribute__((aligned(16))) unsigned short xs[64][LD], ys[NT][64][LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wf = (wave / 2) * 32, wn = (wave % 2) * 32;
  const int r = lane % 16, q = lane / 16;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t f0 = tile / tiles_n * 64, n0 = tile % tiles_n * 64;
    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int xf = tid / 4, xt = tid % 4 * 8;  // staging: a feature's 8 tokens
    const int yn = tid % 64, yt = tid / 64 * 8;  // a column's 8 tokens
    for (int64_t t0 = 0; t0 < p.T; t0 += BLOCK) {
      u32x4 xv = {0u, 0u, 0u, 0u};
      if (f0 + xf < p.F) {
        const int64_t f = f0 + xf;
        const u32x2 w = *reinterpret_cast<const u32x2*>(p.x.codes + f * p.x.ldq + t0 + xt);
        xv = decode8(w, scale_float(p.x.scales[f * p.x.lds + t0 / BLOCK]));
      }
      *reinterpret_cast<u32x4*>(&xs[xf][xt]) = xv;
      unsigned short terms[8][NT];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t t = t0 + yt + i, n = n0 + yn;
        const bool in = t < p.T && n < p.N;
        split_terms<YT>(in ? read_as_float<YT>(p.dY, t * p.ldy + n) : 0.f, terms[i]);
      }
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = terms[2 * i][k] | ((unsigned)terms[2 * i + 1][k] << 16);
        *reinterpret_cast<u32x4*>(&ys[k][yn][yt]) = v;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        h16x8_t xa[2], yb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          xa[i] = *reinterpret_cast<const h16x8_t*>(&xs[wf + 16 * i + r][8 * q]);
          yb[i] = *reinterpret_cast<const h16x8_t*>(&ys[k][wn + 16 * i + r][8 * q]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma16<true>(yb[j], xa[i], acc[i][j]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t f = f0 + wf + 16 * i + r, n = n0 + wn + 16 * j + 4 * q;
        if (f < p.F && n < p.N) store4<CT>(p, f, n, acc[i][j]);
      }
  }
}

// dY as bfloat16 terms: plane k of `terms` holds term k of every value, T
// rows of `ld` columns (N rounded up to 8; the rest zeros).
template <int YT>
__global__ void __launch_bounds__(256)
split_planes(const void* dY, int64_t ldy, int64_t T, int N, int groups, unsigned short* out, int64_t plane) {
  constexpr int NT = kTerms<YT>;
  const int64_t total = T * groups;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / groups;
    const int g = (int)(i - t * groups);
    unsigned short terms[8][NT];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int n = 8 * g + e;
      split_terms<YT>(n < N ? read_as_float<YT>(dY, t * ldy + n) : 0.f, terms[e]);
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = terms[2 * e][k] | ((unsigned)terms[2 * e + 1][k] << 16);
      *reinterpret_cast<u32x4*>(out + k * plane + (t * groups + g) * 8) = v;
    }
  }
}

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
//    byte.  (With 8 bytes a step, tokens 32j + 8q, those reads took 6 LDS
//    cycles each, 4 of them in bank conflicts; 8192 tokens, 4096 x 4096:
//    214 us.)
//  * dY's operands want token-contiguous values of a column: the transpose
//    read ds_read_b64_tr_b16 (in each group of 16 lanes, lane j gets element
//    j%4 of the 8-byte pieces that lanes j/4 + 4t point at).  Its rows'
//    16-byte chunks are XORed by 4(k%4) + (k/8)%2, so that the rows and
//    k runs of one read hit distinct banks.
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

struct PipeArgs {
  Coded x;
  const uint16_t* y;  // bfloat16 planes
  int64_t ldy, plane;
  void* C;            // dW, or the first partial sum
  int64_t ldc, c_stride;
  int T, F, N, terms, chunk;
  float alpha, beta;
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
wgrad_pipe(PipeArgs p, TileMap map, int vec) {
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

// dW = alpha * (sum over splits of partial) + beta * dW, added in order;
// partial rows of `ld` (a multiple of 4) columns, four a thread.
template <int CT>
__global__ void __launch_bounds__(256)
reduce_partials(const float* partial, int64_t ld, int64_t stride, int splits, void* dW, int64_t ldw, int64_t F, int N,
                float alpha, float beta) {
  typedef typename TypeOf<CT>::type T;
  typedef T t4 __attribute__((ext_vector_type(4)));
  const int64_t quads = ld / 4, total = F * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t f = i / quads;
    const int n = 4 * (int)(i - f * quads);
    const float* src = partial + f * ld + n;
    f32x4 v = *reinterpret_cast<const f32x4*>(src);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(src + s * stride);
    T* c = static_cast<T*>(dW) + f * ldw + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] *= alpha;
      if (beta != 0.f && n + e < N) v[e] = __builtin_fmaf(beta, (float)c[e], v[e]);
    }
    if (n + 4 <= N && ((uintptr_t)c & (sizeof(t4) - 1)) == 0) {
      *reinterpret_cast<t4*>(c) = t4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) c[e] = (T)v[e];
    }
  }
}

template <int CT, class S>
hipError_t launch_pipe(const PipeArgs& a, int splits, hipStream_t stream) {
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

template <int CT>
hipError_t launch_tile(int tile, const PipeArgs& a, int splits, hipStream_t stream) {
  return tile == 256 ? launch_pipe<CT, Tile<256, 256, 128, 128>>(a, splits, stream)
                     : launch_pipe<CT, Tile<128, 128, 64, 64>>(a, splits, stream);
}

template <int YT, int CT>
hipError_t launch_planned(const WgradArgs& a, const WgradPlan& w, hipStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  PipeArgs p{a.x, static_cast<const uint16_t*>(a.dY), a.ldy, 0, a.dW, a.ldw, 0, a.T, a.F, a.N, 1, w.chunk, a.alpha, a.beta};
  if (w.planes > 0) {
    const int groups = (a.N + 7) / 8;
    p.y = reinterpret_cast<uint16_t*>(ws);
    p.ldy = 8 * (int64_t)groups;
    p.plane = p.ldy * a.T;
    p.terms = kTerms<YT>;
    const int64_t wgs = ((int64_t)a.T * groups + 255) / 256;
    hipLaunchKernelGGL((split_planes<YT>), dim3((unsigned)(wgs < 8192 ? wgs : 8192)), dim3(256), 0, stream, a.dY, a.ldy,
                       (int64_t)a.T, a.N, groups, reinterpret_cast<unsigned short*>(ws), p.plane);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (w.splits <= 1) return launch_tile<CT>(w.tile, p, 1, stream);
  float* partial = reinterpret_cast<float*>(ws + w.planes);
  p.C = partial;
  p.ldc = ((int64_t)a.N + 3) / 4 * 4;
  p.c_stride = p.ldc * a.F;
  p.alpha = 1.f;
  p.beta = 0.f;
  const hipError_t e = launch_tile<GEMM_DTYPE_F32>(w.tile, p, w.splits, stream);
  if (e != hipSuccess) return e;
  const int64_t wgs = (p.c_stride / 4 + 255) / 256;
  hipLaunchKernelGGL((reduce_partials<CT>), dim3((unsigned)(wgs < 8192 ? wgs : 8192)), dim3(256), 0, stream, partial, p.ldc,
                     p.c_stride, w.splits, a.dW, a.ldw, (int64_t)a.F, a.N, a.alpha, a.beta);
  return hipGetLastError();
}

template <int YT, int CT>
hipError_t launch_general(const WgradArgs& a, hipStream_t stream) {
  const int tiles_n = (a.N + 63) / 64;
  const int64_t tiles = (int64_t)tiles_n * ((a.F + 63) / 64);
  const int64_t most = 1 << 22;  // work-items of a grid: below 2^32
  hipLaunchKernelGGL((wgrad_general<YT, CT>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, stream, a,
                     tiles_n, tiles);
  return hipGetLastError();
}

template <int YT, int CT>
hipError_t launch(const WgradArgs& a, hipStream_t stream) {
  const WgradPlan w = wgrad_plan(YT, a.T, a.F, a.N);
  const bool room = w.bytes() == 0 || (a.workspace && a.workspace_bytes >= w.bytes());
  // What the pipelined kernel takes: scales in 4-byte words, a tile's rows
  // within 31 bits, dY's rows (where they are read as they are) 16-byte
  // aligned.
  const int64_t far = (int64_t)0x7fffffff / 256 - 4096;
  const bool aligned = w.planes > 0 || ((uintptr_t)a.dY % 16 == 0 && a.ldy % 8 == 0);
  if (w.tile == 0 || !room || !aligned || (uintptr_t)a.x.scales % 4 != 0 || a.x.lds % 4 != 0 || a.x.ldq >= far ||
      a.x.lds >= far || a.N >= far || (w.planes == 0 && a.ldy >= far) || a.ldw >= far / 4)
    return launch_general<YT, CT>(a, stream);
  return launch_planned<YT, CT>(a, w, stream);
}

template <int YT>
hipError_t launch(int c_dtype, const WgradArgs& a, hipStream_t stream) {
  return c_dtype == GEMM_DTYPE_F32   ? launch<YT, GEMM_DTYPE_F32>(a, stream)
         : c_dtype == GEMM_DTYPE_F16 ? launch<YT, GEMM_DTYPE_F16>(a, stream)
                                     : launch<YT, GEMM_DTYPE_BF16>(a, stream);
}

}  // namespace

// The pipelined kernel's plan: the tile and the number of token chunks of
// the least modelled time.  Microseconds on MI355X, measured with the card
// full: a slice (64 tokens) of a 256 x 256 tile 1.2 on an idle card to 1.7
// on a full one, of a 128 x 128 tile 0.56 for each that shares a CU; a launch 4; the
// partial sums, written and read, 8 TB/s.  (8192 tokens, 4096 x 4096: 214 us
// on one 256 x 256 tile a CU, 288 on 128 x 128 ones; 16384 tokens, 1024 x
// 1024: 51 us in 8 chunks, 152 in one.)
WgradPlan wgrad_plan(int y_dtype, int64_t T, int64_t F, int64_t N) {
  WgradPlan best;
  const int64_t cap = (int64_t)1 << 23;  // workgroups of a grid, and columns within a tile's 31 bits
  // One block of tokens or less: the general kernel's one launch (16 tokens,
  // 1024 x 1024: 4.8 us against 7.2).
  if (T <= BLOCK || F <= 0 || N <= 0 || N >= cap || F >= cap * 128) return best;
  const int terms = y_dtype == GEMM_DTYPE_BF16 ? 1 : y_dtype == GEMM_DTYPE_F16 ? 2 : 3;
  const double plane = (double)F * (double)((N + 3) / 4 * 16);
  double least = 1e30;
  for (int tile = 128; tile <= 256; tile += 128) {
    const int64_t tiles = ((F + tile - 1) / tile) * ((N + tile - 1) / tile);
    if (tiles >= cap) continue;
    for (int s = 1; s <= 32; ++s) {
      if (s > 1 && (tiles * s > 1024 || plane * s > (double)(1 << 30))) break;
      const int64_t chunk = ((T + s - 1) / s + 127) / 128 * 128;
      if ((T + chunk - 1) / chunk != s) continue;  // fewer chunks than s: seen already
      const double slices = (double)(chunk / 64) * terms;
      const double wgs = (double)(tiles * s), per_cu = (double)((tiles * s + 255) / 256);
      const double slice = tile == 256 ? 1.2 + 0.5 * (wgs < 256 ? wgs / 256 : 1.) : 0.56;
      const double us = 4 + per_cu * slices * slice + (s > 1 ? 4 + 2 * plane * s / 8e6 : 0.);
      if (us < least) {
        least = us;
        best.tile = tile;
        best.splits = s;
        best.chunk = (int)(chunk > 0x7fffff80 ? 0x7fffff80 : chunk);
      }
    }
  }
  if (best.tile == 0) return best;
  if (terms > 1 || N % 8 != 0) best.planes = terms * T * ((N + 7) / 8) * 16;
  if (best.splits > 1) best.partials = (int64_t)best.splits * F * ((N + 3) / 4) * 16;
  return best;
}

hipError_t launch_wgrad(int y_dtype, int c_dtype, const WgradArgs& a, hipStream_t stream) {
  if (a.F <= 0 || a.N <= 0) return hipSuccess;
  return y_dtype == GEMM_DTYPE_F32   ? launch<GEMM_DTYPE_F32>(c_dtype, a, stream)
         : y_dtype == GEMM_DTYPE_F16 ? launch<GEMM_DTYPE_F16>(c_dtype, a, stream)
                                     : launch<GEMM_DTYPE_BF16>(c_dtype, a, stream);
}

}  // namespace mx
}  // namespace gemm

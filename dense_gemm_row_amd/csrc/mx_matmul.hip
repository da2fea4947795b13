// Product of two E2M1 (MXFP4) matrices, C = act(alpha A Bt^T + beta C + bias)
// (include/gemm_mx.h), on v_mfma_scale_f32_16x16x128_f8f6f4.
//
// The instruction multiplies 128 k values of 16 rows by 16 columns: lane l
// holds row l%16's 32 values of k block l/16 (16 bytes of codes) and that
// block's scale byte, which is exactly the storage format, so codes and
// scales go from memory to the matrix core without a conversion.  The
// operands are swapped (the result is C^T's block): register i of lane l is
// then C[l%16][4(l/16) + i], four consecutive columns of one row.
#include "mx_encode.h"
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
        for (int j = 0; j < NT; ++j) {
          b[u][j] = live ? *reinterpret_cast<const i32x4*>(bc[j] + (int64_t)block * 16) : i32x4{0, 0, 0, 0};
          sb[u][j] = live ? bs[j][block] : 127;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          a[u][i] = live ? *reinterpret_cast<const i32x4*>(ac[i] + (int64_t)block * 16) : i32x4{0, 0, 0, 0};
          sa[u][i] = live ? as[i][block] : 127;
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
  hipLaunchKernelGGL((matmul_direct<DT, MT, NT, W, U>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(64 * W),
                     0, stream, a, tiles_n, tiles);
  return hipGetLastError();
}

// Up to 16 rows: 16 columns a workgroup, its W waves taking turns along k,
// four steps (512 k) each, all of whose loads are issued at once.  The
// operand layout has four lanes a row, 64 bytes of it per load, which the
// memory serves badly (16 x 11008 x 4096: 14 us against 10); so the weights'
// codes go through LDS, copied 256 bytes of a row at a time (LDS-direct,
// wave-private, chunk c of row r at c ^ r: conflict-free reads), and their
// scales, 16 bytes of a row, with one copy.  What lies outside the matrix
// reads zeros.  The waves' sums meet in LDS in wave order.
//
// AT >= 0: A is X, values of that type.  A wave reads its 512 k of a row with
// one load a lane, eight values, and encodes them as quantize_rows does, into
// the same LDS layout.  Every workgroup does that for the whole of X, which
// its 16 rows at most keep small beside the weights, and saves the launch
// that would write and the loads that would read the codes.  (Rows past M
// are left as they are: a row of A reaches its own row of C only.)
constexpr int kSkinnyWaves = 8, kSkinnyDepth = 4;

template <int DT, int AT, int W>
__global__ void __launch_bounds__(64 * W)
matmul_skinny(MatmulArgs p) {
  constexpr int U = kSkinnyDepth;
  constexpr int VT = AT < 0 ? 0 : AT, VB = kBytes<VT>;
  __shared__ __attribute__((aligned(1024))) uint8_t codes[W][4096], scales[W][256];
  __shared__ __attribute__((aligned(1024))) uint8_t x_codes[W][AT >= 0 ? 4096 : 16], x_scales[W][AT >= 0 ? 256 : 16];
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane % 16, q = lane / 16;
  const int nb = (p.K + BLOCK - 1) / BLOCK;
  const int steps = (nb + 3) / 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int range = 0x7fffffff;
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b.codes + n0 * p.b.ldq, range);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.b.scales + n0 * p.b.lds, range);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(AT >= 0 ? static_cast<const uint8_t*>(p.X) : p.a.codes, range);
  const __amdgpu_buffer_rsrc_t ras = make_rsrc(p.a.scales, range);
  // Copies: codes of rows 4i + lane/16, scales of row lane/4.
  unsigned ob[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * i + lane / 16;
    ob[i] = n0 + row < p.N ? (unsigned)(row * (int)p.b.ldq) : OOB;
  }
  const unsigned os = n0 + lane / 4 < p.N ? (unsigned)(lane / 4 * (int)p.b.lds) : OOB;
  const unsigned oa = r < p.M ? (unsigned)(r * (int)p.a.ldq) : OOB;
  const unsigned oas = r < p.M ? (unsigned)(r * (int)p.a.lds) : OOB;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = wave * U; s0 < steps; s0 += W * U) {
    i32x4 a[U];
    int sa[U];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int block = 4 * s0 + (lane % 16 ^ (4 * i + lane / 16));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(codes[wave] + 1024 * i), 16,
                                               block < nb ? ob[i] + 16 * block : OOB, 0, 0, 0);
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)scales[wave], 4,
                                             4 * (s0 + lane % 4) < nb ? os + 4 * (s0 + lane % 4) : OOB, 0, 0, 0);
    if constexpr (AT < 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int block = 4 * (s0 + u) + q;
        const bool live = block < nb;
        a[u] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, live ? oa + 16 * block : OOB, 0, 0));
        sa[u] = (int)((unsigned)__builtin_amdgcn_raw_buffer_load_b32(ras, live ? oas + 4 * (s0 + u) : OOB, 0, 0) >> (8 * q));
      }
    } else {
      constexpr int G = AT == GEMM_DTYPE_F32 ? 4 : 8;  // rows in registers at a time
      const int c = 128 * s0 + 8 * lane, left = p.K - c;  // this lane's eight columns
      for (int g = 0; g < p.M; g += G) {
        Eight<VT> v[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
#pragma unroll
          for (int h = 0; h < Eight<VT>::W / 4; ++h) {
            const unsigned at = value_load<VB>(g + i, p.M, (unsigned)(p.ldx * VB), c, left, h);
            const u32x4 x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, at, 0, 0));
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i].w[4 * h + e] = x[e];
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          if (left < 8) {  // past K: zeros
#pragma unroll
            for (int e = 0; e < Eight<VT>::W; ++e) {
              if constexpr (AT == GEMM_DTYPE_F32)
                v[i].w[e] = e < left ? v[i].w[e] : 0u;
              else
                v[i].w[e] = 2 * e + 1 < left ? v[i].w[e] : 2 * e < left ? v[i].w[e] & 0xffffu : 0u;
            }
          }
          const unsigned s = quad_scale<GEMM_MX_E2M1>(v[i]);
          const u32x2 w = encode8<GEMM_MX_E2M1>(v[i], s);
          const int row = (g + i) % 16;
          *reinterpret_cast<unsigned*>(x_codes[wave] + 256 * row + 16 * ((lane / 4) ^ row) + 4 * (lane % 4)) = w[0];
          if (lane % 4 == 0) x_scales[wave][16 * row + lane / 4] = (uint8_t)s;
        }
      }
    }
    // This wave's copies have landed (the compiler takes a copy for a write
    // of its first bytes only, so it has to be told).
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = 256 * r + 16 * ((4 * u + q) ^ r);
      const i32x4 b = *(const lds_i32x4*)(codes[wave] + at);
      const int sb = *(const lds_u8*)(scales[wave] + 16 * r + 4 * u + q);
      if constexpr (AT >= 0) {
        a[u] = *(const lds_i32x4*)(x_codes[wave] + at);
        sa[u] = *(const lds_u8*)(x_scales[wave] + 16 * r + 4 * u + q);
      }
      // (A row's scale bytes past its blocks may be anything.)
      acc = mfma_fp4(b, 4 * (s0 + u) + q < nb ? sb : 0, a[u], sa[u], acc);
    }
    // The next turn's copies and codes wait for these reads.
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
  }
  // (The sums take the codes' place: each wave's own, until the barrier.)
  *reinterpret_cast<f32x4*>(codes[wave] + 64 * r + 16 * q) = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int m = threadIdx.x / 4, n = threadIdx.x % 4 * 4;
    f32x4 v = *reinterpret_cast<const f32x4*>(codes[0] + 64 * m + 4 * n);
#pragma unroll
    for (int w = 1; w < W; ++w) v += *reinterpret_cast<const f32x4*>(codes[w] + 64 * m + 4 * n);
    if (m < p.M && n0 + n < p.N) store4<DT>(p, m, n0 + n, v);
  }
#endif
}

// What it takes: 16 rows of every operand within 31 bits, scales in 4-byte
// words, and (values) rows of whole 16 bytes.
template <int AT>
bool skinny_ok(const MatmulArgs& a) {
  const int64_t far = 1 << 26;
  if (a.K <= 0 || a.M > 16 || a.N > (int64_t)16 << 22 || a.b.ldq >= far || a.b.lds >= far || a.b.lds % 4 != 0 ||
      (uintptr_t)a.b.scales % 4 != 0)
    return false;
  if constexpr (AT < 0)
    return a.a.ldq < far && a.a.lds < far && a.a.lds % 4 == 0 && (uintptr_t)a.a.scales % 4 == 0;
  else
    return (uintptr_t)a.X % 16 == 0 && a.ldx * kBytes<AT> % 16 == 0 && a.ldx * kBytes<AT> < far;
}

template <int DT, int AT>
hipError_t launch_skinny(const MatmulArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 15) / 16));
  // One turn of every wave, where 16 can do it.
  if (a.K > 128 * kSkinnyDepth * kSkinnyWaves)
    hipLaunchKernelGGL((matmul_skinny<DT, AT, 16>), grid, dim3(64 * 16), 0, stream, a);
  else
    hipLaunchKernelGGL((matmul_skinny<DT, AT, kSkinnyWaves>), grid, dim3(64 * kSkinnyWaves), 0, stream, a);
  return hipGetLastError();
}

// The pipelined kernel: a workgroup of four waves computes BM x BN, each
// wave WM x WN in 16 x 16 blocks, 256 k (128 bytes a row) per slice through
// two LDS stages.
//  * Codes go from memory to LDS with 16-byte LDS-direct copies.  A 16-byte
//    read serves 16 lanes at a time, rows 0-3 and 12-15 of an even lane group
//    with rows 4-11 of the next (or the other way round); with step j's chunk
//    of group q at position (4j + q) ^ (r/2)%8 of row r's 128 bytes, those
//    hit distinct banks.
//  * Scales go to LDS for two slices at a time, 16 bytes of a row (SC = 16:
//    one copy a wave and operand; SC = 4, for scale rows that are only 4-byte
//    aligned, four).  A slice's two steps take blocks 2q and 2q + 1 for lane
//    group q, so that a lane's scales for both come with one read (of the
//    word that two groups share), and the instruction picks the byte.  A
//    bit-field extraction takes them out of the word and clears those past
//    the matrix' blocks, which may be anything (255 would be NaN).
//    (8192^3: 273 us with 8 bytes a slice in 4-byte copies and a byte read
//    for each step.)
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

template <int DT, class S>
hipError_t launch_pipe_tile(const MatmulArgs& a, hipStream_t stream) {
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

template <int DT, int BM, int BN, int WM, int WN>
hipError_t launch_pipe(const MatmulArgs& a, hipStream_t stream) {
  const bool wide = (((uintptr_t)a.a.scales | (uintptr_t)a.b.scales) % 16 | (a.a.lds | a.b.lds) % 16) == 0;
  return wide ? launch_pipe_tile<DT, Tile<BM, BN, WM, WN, 16>>(a, stream)
              : launch_pipe_tile<DT, Tile<BM, BN, WM, WN, 4>>(a, stream);
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
  if (a.M <= 16)
    return skinny_ok<-1>(a) ? launch_skinny<DT, -1>(a, stream)
                            : launch_direct<DT, 1, 1, kSkinnyWaves, kSkinnyDepth>(a, stream);
  if (!pipe_ok(a)) return launch_direct<DT, 4, 4, 4, 1>(a, stream);
  // 256 x 256 tiles reuse each operand byte twice as often, 128 x 128 ones
  // fill the 256 CUs with a quarter of the outputs (4096^3: 39 against
  // 50 us; 2048^3: 19 against 10 us).
  const int64_t tiles = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  if (tiles >= 192) return launch_pipe<DT, 256, 256, 128, 128>(a, stream);
  return launch_pipe<DT, 128, 128, 64, 64>(a, stream);
}

}  // namespace

bool values_fit(int a_dtype, const MatmulArgs& a) {
  return a_dtype == GEMM_DTYPE_F32   ? skinny_ok<GEMM_DTYPE_F32>(a)
         : a_dtype == GEMM_DTYPE_F16 ? skinny_ok<GEMM_DTYPE_F16>(a)
                                     : skinny_ok<GEMM_DTYPE_BF16>(a);
}

hipError_t launch_matmul_values(int a_dtype, int c_dtype, const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  auto with = [&](auto DT) {
    constexpr int D = decltype(DT)::value;
    return a_dtype == GEMM_DTYPE_F32   ? launch_skinny<D, GEMM_DTYPE_F32>(a, stream)
           : a_dtype == GEMM_DTYPE_F16 ? launch_skinny<D, GEMM_DTYPE_F16>(a, stream)
                                       : launch_skinny<D, GEMM_DTYPE_BF16>(a, stream);
  };
  return c_dtype == GEMM_DTYPE_F32   ? with(IC<GEMM_DTYPE_F32>{})
         : c_dtype == GEMM_DTYPE_F16 ? with(IC<GEMM_DTYPE_F16>{})
                                     : with(IC<GEMM_DTYPE_BF16>{});
}

hipError_t launch_matmul(int c_dtype, const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 0 || a.N <= 0) return hipSuccess;
  return c_dtype == GEMM_DTYPE_F32   ? launch<GEMM_DTYPE_F32>(a, stream)
         : c_dtype == GEMM_DTYPE_F16 ? launch<GEMM_DTYPE_F16>(a, stream)
                                     : launch<GEMM_DTYPE_BF16>(a, stream);
}

}  // namespace mx
}  // namespace gemm

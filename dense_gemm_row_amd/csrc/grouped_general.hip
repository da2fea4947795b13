// The grouped products for any operands: every type, alignment, stride and
// size.  A workgroup of four waves computes a SIDE x SIDE tile (128 or 64), 128
// bytes of k per slice (64 values of 16 bits, 32 of 32), each wave a quarter in
// blocks of the 16 x 16 matrix instruction (FP32: k 4, binary16 and bfloat16: k
// 32), FP32 accumulation.
//  * Operands go through registers, in 16-byte pieces wherever they begin
//    (global loads need no alignment): what lies past the end of a row is cut
//    off a piece that ends there, so nothing outside an operand is read.  Two
//    slices are on their way in registers while a third is multiplied.
//  * LDS holds two stages.  ALONG (k contiguous: X; W given transposed): rows
//    of 128 bytes, 16-byte chunks XORed by (row / 2) % 8; an operand is one
//    16-byte read.  ACROSS (rows contiguous, k down the rows: W; both of the
//    gradient's): a row for each k, chunks XORed so that an operand's reads
//    (16 bits: two transpose reads; FP32: four values) meet distinct banks.
//  * The matrix instruction gets the operands swapped, so that a lane holds
//    four consecutive columns of one row of the result.
// Rows and columns past an operand's end are copies of others and not stored;
// k past the end counts as zero.  64-bit addresses throughout.
#include <type_traits>
#include <utility>

#include "grouped_internal.h"
#include "mx_pipe.h"

namespace gemm {
namespace grouped {
namespace {

constexpr int THREADS = 256;

template <int DT>
struct TypeOf;
template <>
struct TypeOf<GEMM_DTYPE_F32> { typedef float type; };
template <>
struct TypeOf<GEMM_DTYPE_F16> { typedef _Float16 type; };
template <>
struct TypeOf<GEMM_DTYPE_BF16> { typedef __bf16 type; };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

template <class T>
struct Operand {
  const T* at;  // element (0, 0) of the tile
  int64_t ld;
  int rows;     // rows (columns of the result) from the tile on
  int total;    // and in all
};

// A piece without its first n values (of `size` bytes), zeros behind.
__device__ __forceinline__ i32x4 without(i32x4 v, int n, int size) {
  const unsigned __int128 bits = __builtin_bit_cast(unsigned __int128, v);
  return n * size >= 16 ? i32x4{0, 0, 0, 0} : __builtin_bit_cast(i32x4, bits >> (8 * size * n));
}

// One operand's WIDTH rows of a slice: this thread's pieces of it, on their way
// from memory to LDS, and the operands that a lane reads there.  Its pieces
// are the same chunk of rows (ACROSS: of k) STEP apart.
template <class T, bool ACROSS, int WIDTH>
struct Panel {
  static constexpr int ES = sizeof(T), PER = 16 / ES, BK = 128 / ES, N = WIDTH * 128 / 16 / THREADS, BYTES = 128 * WIDTH;
  static constexpr int CHUNKS = ACROSS ? WIDTH / PER : 8, STEP = THREADS / CHUNKS;
  const T* at[ACROSS ? 1 : N];  // pieces of the slice at k 0
  int64_t ld;
  int K, rows, first, cut;  // (the first one's k; values before it in its 16 bytes)
  bool edge, tiny;
  __device__ static __forceinline__ int row0() { return (int)threadIdx.x / CHUNKS; }
  __device__ static __forceinline__ int chunk() { return (int)threadIdx.x % CHUNKS; }
  // Chunk c of LDS row `row` (ACROSS: of k, otherwise of a row).
  __device__ static constexpr int place(int row, int c) {
    if constexpr (!ACROSS) return 128 * row + 16 * (c ^ (row / 2 % 8));
    else if constexpr (ES == 4) return 16 * CHUNKS * row + 16 * (c ^ (4 * (row / 4 % 4)));
    else if constexpr (CHUNKS >= 16) return 16 * CHUNKS * row + 16 * (c ^ (4 * (row % 4)) ^ (2 * (row / 8 % 2)));
    else return 16 * CHUNKS * row + 16 * (c ^ (2 * (row / 2 % 2)) ^ (4 * (row / 8 % 2)));
  }
  __device__ __forceinline__ Panel(const Operand<T>& o, int K_) : ld(o.ld), K(K_), rows(o.rows), cut(0) {
    edge = ACROSS && rows < WIDTH;
    tiny = ACROSS ? o.total < PER : K < PER;  // (no whole piece in a row)
    if constexpr (ACROSS) {
      first = row0();
      const int n = PER * chunk();
      if (!tiny) cut = piece_early(rows - n, PER);
      at[0] = o.at + row0() * ld + (n - cut);
    } else {
      first = PER * chunk();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = row0() + i * STEP;
        at[i] = o.at + (r < rows ? r : rows - 1) * ld + first;
      }
    }
  }
  // The slice at k0, which is whole, or (EDGE) any.
  template <bool EDGE>
  __device__ __forceinline__ void fetch(int64_t k0, i32x4 (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T* p = ACROSS ? at[0] + (k0 + i * STEP) * ld : at[i] + k0;
      if constexpr (!EDGE) {
        __builtin_memcpy(&v[i], p, 16);
      } else {
        v[i] = i32x4{0, 0, 0, 0};
        const int64_t left = K - (k0 + first + (ACROSS ? i * STEP : 0));
        if (left <= 0) continue;
        if (tiny) {
          T e[PER];
#pragma unroll
          for (int u = 0; u < PER; ++u) e[u] = (ACROSS ? PER * chunk() + u < rows : u < left) ? p[u] : (T)0.f;
          __builtin_memcpy(&v[i], e, 16);
        } else {
          const int gone = ACROSS ? 0 : piece_early(left, PER);
          __builtin_memcpy(&v[i], p - gone, 16);
          v[i] = without(v[i], gone, ES);
        }
      }
    }
  }
  __device__ __forceinline__ void store(uint8_t* stage, i32x4 (&v)[N]) const {
    if (ACROSS && edge) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = without(v[i], cut, ES);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<i32x4*>(stage + place(row0() + i * STEP, chunk())) = v[i];
  }
  // The operand of rows row0 .. + 15 in step j (half of the slice's k): for 16
  // bits lane l's k 32j + 8 (l / 16) .. + 7, for FP32 k 16j + 4 (l / 16) .. + 3.
  __device__ static __forceinline__ i32x4 operand(const uint8_t* stage, int row0, int j) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int l = threadIdx.x & 63, r = l % 16, q = l / 16;
    if constexpr (!ACROSS) {
      return *reinterpret_cast<const i32x4*>(stage + place(row0 + r, 4 * j + q));
    } else if constexpr (ES == 4) {
      i32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = *reinterpret_cast<const int*>(stage + place(16 * j + 4 * q + e, (row0 + r) / 4) + 4 * (r % 4));
      return v;
    } else {
      // (In each group of 16 lanes, lane r gets element r % 4 of the 8-byte
      // pieces that lanes r / 4 + 4t point at.)
      const uint8_t* p = stage + place(32 * j + 8 * q + r / 4, (row0 + 4 * (r % 4)) / 8) + 8 * (r % 2);
      const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx::lds_s16x4*)p));
      const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((mx::lds_s16x4*)(p + 4 * 16 * CHUNKS)));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3);
    }
#else
    return i32x4{0, 0, 0, 0};
#endif
  }
};

// acc[j][i], register e of lane l: row 16i + l%16, column 16j + 4(l/16) + e
// of the wave's share (row (wave/2), column (wave%2)), SIDE / 2 square.
template <int DT, bool AX, bool BX, int SIDE>
__device__ __forceinline__ void tile_sums(const Operand<typename TypeOf<DT>::type>& A,
                                          const Operand<typename TypeOf<DT>::type>& B, int K, f32x4 (&acc)[SIDE / 32][SIDE / 32]) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename TypeOf<DT>::type T;
  typedef Panel<T, AX, SIDE> PA;
  typedef Panel<T, BX, SIDE> PB;
  constexpr int BK = PA::BK, NB = SIDE / 32, DEPTH = SIDE == 128 ? 1 : 2;
  __shared__ __attribute__((aligned(16))) uint8_t la[2][PA::BYTES], lb[2][PB::BYTES];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), m0 = SIDE / 2 * (wave / 2), n0 = SIDE / 2 * (wave % 2);
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (K <= 0) return;
  const PA a(A, K);
  const PB b(B, K);
  i32x4 ra[DEPTH][PA::N], rb[DEPTH][PB::N];
  const int slices = (int)(((int64_t)K + BK - 1) / BK), whole = a.tiny || b.tiny ? 0 : K / BK;
  auto fetch = [&](int i, auto EDGE, auto R) __attribute__((always_inline)) {
    a.template fetch<decltype(EDGE)::value>((int64_t)i * BK, ra[decltype(R)::value]);
    b.template fetch<decltype(EDGE)::value>((int64_t)i * BK, rb[decltype(R)::value]);
  };
  // Slice i from its stage; the next one, which has landed, goes into the
  // other; the third from it sets out.  (The barrier does not wait for loads.)
  auto step = [&](int i, auto R, auto EDGE) __attribute__((always_inline)) {
    constexpr int c = decltype(R)::value, n = 1 - c;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      i32x4 x[NB], w[NB];
#pragma unroll
      for (int u = 0; u < NB; ++u) x[u] = PA::operand(la[c], m0 + 16 * u, j);
#pragma unroll
      for (int u = 0; u < NB; ++u) w[u] = PB::operand(lb[c], n0 + 16 * u, j);
#pragma unroll
      for (int v = 0; v < NB; ++v)
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          if constexpr (DT == GEMM_DTYPE_F32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[v][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(f32x4, w[v])[e], __builtin_bit_cast(f32x4, x[u])[e],
                                                               acc[v][u], 0, 0, 0);
          } else {
            acc[v][u] = mfma16<DT == GEMM_DTYPE_BF16>(__builtin_bit_cast(h16x8_t, w[v]), __builtin_bit_cast(h16x8_t, x[u]), acc[v][u]);
          }
        }
    }
    a.store(la[n], ra[n % DEPTH]);
    b.store(lb[n], rb[n % DEPTH]);
    fetch(i + 1 + DEPTH, EDGE, std::integral_constant<int, n % DEPTH>{});
  };
  constexpr std::integral_constant<int, 0> R0{};
  constexpr std::integral_constant<int, 1> R1{};
  constexpr std::true_type EDGE{};
  constexpr std::false_type WHOLE{};
  fetch(0, EDGE, R0);
  if constexpr (DEPTH == 2) fetch(1, EDGE, R1);
  __syncthreads();  // (the tile before has been read)
  a.store(la[0], ra[0]);
  b.store(lb[0], rb[0]);
  fetch(DEPTH, EDGE, R0);
  int i = 0;
  static_assert(2 + DEPTH <= 4, "the second step's fetch is of a whole slice");
  for (; i + 4 < whole; i += 2) {
    step(i, R0, WHOLE);
    step(i + 1, R1, WHOLE);
  }
  for (; i < slices; i += 2) {  // (slices past the end are zeros)
    step(i, R0, EDGE);
    step(i + 1, R1, EDGE);
  }
#endif
}

// The lane's results inside rows x cols: f(row, column, four values, how many
// of them are inside).  Lanes r and r + 8 of 16 exchange halves of two blocks,
// so that a call's 64 lanes have 32 columns of eight rows, not 16 of 16.  (64
// groups of 6 rows, gradient of 801 x 1203: 103 us by 16 rows, 97 so.)
template <int SIDE, class F>
__device__ __forceinline__ void each_four(const f32x4 (&acc)[SIDE / 32][SIDE / 32], int rows, int cols, F&& f) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, r = l % 16;
#pragma unroll
  for (int i = 0; i < SIDE / 32; ++i) {
    const int row = SIDE / 2 * (wave / 2) + 16 * i + r % 8;
#pragma unroll
    for (int j = 0; j < SIDE / 32; j += 2) {
      const i32x4 x = __builtin_bit_cast(i32x4, acc[j][i]), y = __builtin_bit_cast(i32x4, acc[j + 1][i]);
      i32x4 upper, lower;
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // (row_ror:8, written to lanes 8 .. 15 and to lanes 0 .. 7)
        upper[e] = __builtin_amdgcn_update_dpp(x[e], y[e], 0x128, 0xf, 0xc, false);
        lower[e] = __builtin_amdgcn_update_dpp(y[e], x[e], 0x128, 0xf, 0x3, false);
      }
      const int col = SIDE / 2 * (wave % 2) + 16 * (j + r / 8) + 4 * (l / 16), left = cols - col;
      if (row < rows && left > 0) f(row, col, __builtin_bit_cast(f32x4, upper), left < 4 ? left : 4);
      if (row + 8 < rows && left > 0) f(row + 8, col, __builtin_bit_cast(f32x4, lower), left < 4 ? left : 4);
    }
  }
#endif
}
// n of four values to (unaligned) memory.
template <class C>
__device__ __forceinline__ void store_four(C* to, f32x4 v, int n) {
  C e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = (C)v[i];
  if (n == 4) {
    __builtin_memcpy(to, e, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) to[i] = e[i];
  }
}

// (A grid has at most 2^22 workgroups; they walk over the tiles.)
constexpr int64_t kMostBlocks = 1 << 22;

// Tile `b` of tiles_m x tiles_n, dealt to the XCDs in runs where an int counts
// them; false: there is none.
__device__ __forceinline__ bool tile_at(int64_t b, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int64_t tiles = (int64_t)tiles_m * tiles_n;
  if (b >= tiles) return false;
  if (tiles < 1ll << 31) {
    tile_of_block((int)b, TileMap{tiles_m, tiles_n, GEMM_ORDER_XCD, 4, kXcds}, tm, tn);
  } else {
    tm = (int)(b / tiles_n);
    tn = (int)(b % tiles_n);
  }
  return true;
}

template <int DT, int CT, bool TRANS, int SIDE>
__global__ void __launch_bounds__(THREADS, 2) matmul_general(MatmulArgs p, int64_t tiles, int tiles_n) {
  typedef typename TypeOf<DT>::type T;
  typedef typename TypeOf<CT>::type C;
  const RowTiles all(p.offsets, p.G, p.T, p.fill, SIDE);
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    int tm, tn;
    if (!tile_at(b, all.count, tiles_n, tm, tn)) return;  // (`tiles` are the most that offsets can give)
    const RowTile t = all.find(tm);
    const int n0 = tn * SIDE, cols = p.N - n0;
    const T* X = static_cast<const T*>(p.X) + t.row0 * p.ldx;
    const T* W = static_cast<const T*>(p.W) + (t.g < 0 ? 0 : t.g) * p.stride_w + (TRANS ? n0 * p.ldw : n0);
    f32x4 acc[SIDE / 32][SIDE / 32];
    // (Rows of no group: a sum over no k.)
    tile_sums<DT, false, !TRANS, SIDE>(Operand<T>{X, p.ldx, t.rows, p.T}, Operand<T>{W, p.ldw, cols, p.N}, t.g < 0 ? 0 : p.K, acc);
    C* Y = static_cast<C*>(p.Y) + t.row0 * p.ldy + n0;
    each_four<SIDE>(acc, t.rows, cols, [&](int row, int col, f32x4 v, int n) { store_four(Y + row * p.ldy + col, v, n); });
  }
}

template <int DT, int CT, int SIDE>
__global__ void __launch_bounds__(THREADS, 2) wgrad_general(WgradArgs p, int64_t tiles, int tiles_k, int tiles_n) {
  typedef typename TypeOf<DT>::type T;
  typedef typename TypeOf<CT>::type C;
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    const int64_t each = (int64_t)tiles_k * tiles_n;
    const int g = (int)(b / each);
    int tm, tn;
    tile_at(b % each, tiles_k, tiles_n, tm, tn);
    const int m0 = tm * SIDE, n0 = tn * SIDE, rows = p.K - m0, cols = p.N - n0;
    int start, end;
    group_rows(p.offsets, p.T, g, start, end);
    f32x4 acc[SIDE / 32][SIDE / 32];
    tile_sums<DT, true, true, SIDE>(Operand<T>{static_cast<const T*>(p.X) + start * p.ldx + m0, p.ldx, rows, p.K},
                                    Operand<T>{static_cast<const T*>(p.dY) + start * p.ldy + n0, p.ldy, cols, p.N}, end - start, acc);
    C* W = static_cast<C*>(p.dW) + g * p.stride_w + m0 * p.ldw + n0;
    each_four<SIDE>(acc, rows, cols, [&](int row, int col, f32x4 v, int n) {
      C* at = W + row * p.ldw + col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] *= p.alpha;
        if (p.beta != 0.f && e < n) v[e] = __builtin_fmaf(p.beta, (float)at[e], v[e]);
      }
      store_four(at, v, n);
    });
  }
}

dim3 grid_of(int64_t tiles) { return dim3((unsigned)(tiles < kMostBlocks ? tiles : kMostBlocks)); }

template <int DT, int CT, int SIDE>
hipError_t on_tile(const MatmulArgs& a, hipStream_t s) {
  const int64_t tiles_n = tiles_along(a.N, SIDE), tiles = most_tiles(a.T, a.G, a.fill, SIDE) * tiles_n;
  if (tiles <= 0) return hipSuccess;
  if (a.trans_w) hipLaunchKernelGGL((matmul_general<DT, CT, true, SIDE>), grid_of(tiles), dim3(THREADS), 0, s, a, tiles, (int)tiles_n);
  else hipLaunchKernelGGL((matmul_general<DT, CT, false, SIDE>), grid_of(tiles), dim3(THREADS), 0, s, a, tiles, (int)tiles_n);
  return hipGetLastError();
}

template <int DT, int CT, int SIDE>
hipError_t on_tile(const WgradArgs& a, hipStream_t s) {
  const int64_t tiles_k = tiles_along(a.K, SIDE), tiles_n = tiles_along(a.N, SIDE), tiles = a.G * tiles_k * tiles_n;
  if (tiles <= 0) return hipSuccess;
  hipLaunchKernelGGL((wgrad_general<DT, CT, SIDE>), grid_of(tiles), dim3(THREADS), 0, s, a, tiles, (int)tiles_k, (int)tiles_n);
  return hipGetLastError();
}

// Tiles of 128 where groups fill them and enough are likely to occupy the GPU;
// for FP32, bound by the matrix instruction, more of 64 are spread more evenly,
// but the gradient's operands, down the rows both, take four reads each.  (16
// bits, 8 groups of 1000 rows, 2001 x 2001: 160 us on 128 and 207 on 64, gradient
// 173 and 226; 64 groups of 47 rows, 801 x 1203: 66 and 52; of 6, gradient 120
// and 103.  FP32, 8 groups of 250 rows, 2048 x 2048: 272 and 203, gradient 204
// and 220.)
bool wide(const MatmulArgs& a) {
  return a.T >= 96ll * a.G && (a.T / 128 + (a.T < a.G ? a.T : a.G) / 2) * tiles_along(a.N, 128) >= 256;
}
bool wide(const WgradArgs& a) { return a.T >= 64ll * a.G && a.G * tiles_along(a.K, 128) * tiles_along(a.N, 128) >= 256; }

template <int DT, int CT, class Args>
hipError_t launch(const Args& a, hipStream_t s) {
  if constexpr (DT == GEMM_DTYPE_F32 && std::is_same_v<Args, MatmulArgs>) return on_tile<DT, CT, 64>(a, s);
  else return wide(a) ? on_tile<DT, CT, 128>(a, s) : on_tile<DT, CT, 64>(a, s);
}

template <class Args>
hipError_t dispatch(int dtype, int c_dtype, const Args& a, hipStream_t s) {
  if (dtype == GEMM_DTYPE_F32) return launch<GEMM_DTYPE_F32, GEMM_DTYPE_F32>(a, s);
  if (dtype == GEMM_DTYPE_F16)
    return c_dtype == GEMM_DTYPE_F32 ? launch<GEMM_DTYPE_F16, GEMM_DTYPE_F32>(a, s) : launch<GEMM_DTYPE_F16, GEMM_DTYPE_F16>(a, s);
  return c_dtype == GEMM_DTYPE_F32 ? launch<GEMM_DTYPE_BF16, GEMM_DTYPE_F32>(a, s) : launch<GEMM_DTYPE_BF16, GEMM_DTYPE_BF16>(a, s);
}

}  // namespace

hipError_t launch_general(int dtype, int c_dtype, const MatmulArgs& a, hipStream_t s) { return dispatch(dtype, c_dtype, a, s); }
hipError_t launch_general(int dtype, int c_dtype, const WgradArgs& a, hipStream_t s) { return dispatch(dtype, c_dtype, a, s); }

}  // namespace grouped
}  // namespace gemm

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
  const int nb = (int)blocks_of(p.K);
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
  const int tiles_n = (int)ceil_div(a.N, 16 * NT);
  const int64_t tiles = tiles_n * ceil_div(a.M, 16 * MT);
  const int64_t most = 1 << 22;  // work-items of a grid: below 2^32
  hipLaunchKernelGGL((matmul_direct<DT, MT, NT, W, U>), dim3((unsigned)(tiles < most ? tiles : most)), dim3(64 * W),
                     0, stream, a, tiles_n, tiles);
  return hipGetLastError();
}

// Up to 16 rows: 16 columns a workgroup, its W waves taking turns along k,
// four steps (512 k) each, all of whose loads are issued at once.  The
// operand layout has four lanes a row, 64 bytes of it per load, which the
// memory serves badly (16 x 11008 x 4096: 14 us against 11); so the weights'
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
// words, fewer than 2^22 workgroups (of up to 1024 work-items: a grid's have
// to stay below 2^32), and (values) rows of whole 16 bytes.
template <int AT>
bool skinny_ok(const MatmulArgs& a) {
  const int64_t far = 1 << 26;
  if (a.K <= 0 || a.M > 16 || a.N > far - 16 || a.b.ldq >= far || a.b.lds >= far || a.b.lds % 4 != 0 ||
      (uintptr_t)a.b.scales % 4 != 0)
    return false;
  if constexpr (AT < 0)
    return a.a.ldq < far && a.a.lds < far && a.a.lds % 4 == 0 && (uintptr_t)a.a.scales % 4 == 0;
  else
    return (uintptr_t)a.X % 16 == 0 && a.ldx * kBytes<AT> % 16 == 0 && a.ldx * kBytes<AT> < far;
}

template <int DT, int AT>
hipError_t launch_skinny(const MatmulArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(a.N, 16));
  // One turn of every wave, where 16 can do it.
  if (a.K > 128 * kSkinnyDepth * kSkinnyWaves)
    hipLaunchKernelGGL((matmul_skinny<DT, AT, 16>), grid, dim3(64 * 16), 0, stream, a);
  else
    hipLaunchKernelGGL((matmul_skinny<DT, AT, kSkinnyWaves>), grid, dim3(64 * kSkinnyWaves), 0, stream, a);
  return hipGetLastError();
}

// The pipelined kernel (mx_matmul_pipe.hip), with scales in 16-byte pieces
// where both operands' rows are whole ones of them.
template <int DT, int SIDE>
hipError_t launch_pipe(const MatmulArgs& a, hipStream_t stream) {
  const bool wide = (((uintptr_t)a.a.scales | (uintptr_t)a.b.scales) % 16 | (a.a.lds | a.b.lds) % 16) == 0;
  return wide ? launch_matmul_pipe<DT, SIDE, 16>(a, stream) : launch_matmul_pipe<DT, SIDE, 4>(a, stream);
}

// What the pipelined kernel takes: scales in 4-byte words, a tile's rows
// within 31 bits, a grid below 2^32 work-items.
bool pipe_ok(const MatmulArgs& a) {
  const int64_t far = (int64_t)0x7fffffff / 256 - 4096;
  return a.K > 0 && (uintptr_t)a.a.scales % 4 == 0 && a.a.lds % 4 == 0 && (uintptr_t)a.b.scales % 4 == 0 &&
         a.b.lds % 4 == 0 && a.a.ldq < far && a.b.ldq < far && a.a.lds < far && a.b.lds < far && a.ldc < far / 4 &&
         ceil_div(a.M, 128) * ceil_div(a.N, 128) < (1 << 23);
}

template <int DT>
hipError_t launch(const MatmulArgs& a, hipStream_t stream) {
  if (a.M <= 16)
    return skinny_ok<-1>(a) ? launch_skinny<DT, -1>(a, stream)
                            : launch_direct<DT, 1, 1, kSkinnyWaves, kSkinnyDepth>(a, stream);
  if (!pipe_ok(a)) return launch_direct<DT, 4, 4, 4, 1>(a, stream);
  // 256 x 256 tiles reuse each operand byte twice as often, 128 x 128 ones
  // fill the 256 CUs with a quarter of the outputs.  Large against small
  // tiles, K = 4096, bfloat16, by the number of large ones: 64 (2048^2) 28
  // against 15.5 us, 100 29 against 22, 144 35 against 40, 196 56 against 64,
  // 256 (4096^2) 37 against 45, 289 102 against 86, 361 102 against 98, 400
  // 80 against 88, 484 70 against 83.  (The border is not at the best place:
  // 144 would do with the large ones, and 257 to about 380 of them, a second
  // and mostly empty round, with the small.)
  const int64_t tiles = ceil_div(a.M, 256) * ceil_div(a.N, 256);
  if (tiles >= 192) return launch_pipe<DT, 256>(a, stream);
  return launch_pipe<DT, 128>(a, stream);
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

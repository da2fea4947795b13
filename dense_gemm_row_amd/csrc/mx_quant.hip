// Quantisation to the microscaled formats and back (include/gemm_mx.h).
//
// A block of 32 values shares the factor 2^e taken from its largest
// magnitude; the elements are x / 2^e rounded to nearest even by the
// conversion instructions (v_cvt_scalef32_pk_fp4_* / _fp8_*; their rounding,
// their saturation and their reading of the factor were checked on the
// device against every grid midpoint).  The largest magnitude is found on
// the bit patterns with the sign cleared: as unsigned integers they are
// ordered like the magnitudes, and infinities and NaN are above all finite
// values, so one maximum also says whether the block holds one.
//
// Both directions are bound by HBM: one pass, each value read once.
// * Along rows, a lane holds 8 consecutive values (a quarter of a block; 16
//   bytes of 16-bit input), and the four lanes of a block exchange maxima
//   by lane permutation.
// * Transposed, a lane holds 32 rows of 16 bytes' worth of columns, whole
//   blocks of its columns, so nothing is exchanged; the transposition is
//   that a lane writes each of its columns' 32 codes as one run.  Four
//   lanes on consecutive row blocks of the same columns make that run 64
//   (E2M1) or 128 bytes (E4M3), sixteen lanes on consecutive column groups
//   make 256-byte reads.
#include "mx_encode.h"

namespace gemm {
namespace mx {
namespace {

constexpr int kThreads = 256;

// Rows: workgroup (rows of `width` lanes) x UNROLL chunks of 8 columns.
template <int DT, int FMT, bool VEC, int UNROLL>
__global__ void __launch_bounds__(kThreads)
quantize_rows(QuantArgs a, int chunks, int width_log2, int tiles_x) {
  constexpr int QB = kBlockBytes<FMT> / 4;  // code bytes of 8 values
  const int width = 1 << width_log2;
  const int tid = threadIdx.x;
  const int ty = blockIdx.x / tiles_x, tx = blockIdx.x - ty * tiles_x;
  const int64_t row = ((int64_t)ty << (8 - width_log2)) + (tid >> width_log2);
  if (row >= a.rows) return;
  const unsigned char* x = static_cast<const unsigned char*>(a.X) + row * a.ldx * kBytes<DT>;
  const int64_t c0 = (int64_t)tx * width * UNROLL + (tid & (width - 1));  // chunk index
  Eight<DT> v[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int64_t c = 8 * (c0 + (int64_t)u * width);
    v[u] = load8<DT, VEC>(x, c, a.cols - c);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int64_t chunk = c0 + (int64_t)u * width;
    const unsigned s = quad_scale<FMT>(v[u]);
    if (chunk >= chunks) continue;
    const u32x2 q = encode8<FMT>(v[u], s);
    uint8_t* dst = a.codes + row * a.ldq + chunk * QB;
    if constexpr (FMT == GEMM_MX_E2M1)
      *reinterpret_cast<unsigned*>(dst) = q[0];
    else
      *reinterpret_cast<u32x2*>(dst) = q;
    if ((tid & 3) == 0) a.scales[row * a.lds + chunk / 4] = (uint8_t)s;
  }
}

// One row of a lane's CPT columns, as words (16-bit types: column pairs).
template <int DT, int CPT>
struct Cols {
  static constexpr int W = DT == GEMM_DTYPE_F32 ? CPT : (CPT + 1) / 2;
  unsigned w[W];
};

// n of the CPT columns exist (the rest are zeros).
template <int DT, int CPT>
__device__ __forceinline__ Cols<DT, CPT> load_cols(const unsigned char* p, int n) {
  Cols<DT, CPT> v;
  if constexpr (CPT > 1) {
    if (n >= CPT) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.w[j] = x[j];
      return v;
    }
  }
#pragma unroll
  for (int i = 0; i < Cols<DT, CPT>::W; ++i) {
    if constexpr (DT == GEMM_DTYPE_F32) {
      v.w[i] = i < n ? reinterpret_cast<const unsigned*>(p)[i] : 0u;
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      v.w[i] = 2 * i < n ? h[2 * i] : 0u;
      if constexpr (CPT > 1) v.w[i] |= (2 * i + 1 < n ? (unsigned)h[2 * i + 1] : 0u) << 16;
    }
  }
  return v;
}

// Transposed: lane (row block rb of RB, column group cg of 64/RB) of a wave
// holds 32 rows x CPT columns.  CPT columns are 16 bytes (VEC), or one.
template <int DT, int FMT, bool VEC, int RB>
__global__ void __launch_bounds__(kThreads)
quantize_cols(QuantArgs a, int nblocks, int tiles_x) {
  constexpr int CPT = VEC ? 16 / kBytes<DT> : 1;
  constexpr int CG = 64 / RB;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ty = blockIdx.x / tiles_x, tx = blockIdx.x - ty * tiles_x;
  const int64_t c0 = ((int64_t)tx * 4 + wave) * (CG * CPT) + (lane / RB) * CPT;
  const int64_t rb = (int64_t)ty * RB + lane % RB;
  if (c0 >= a.cols || rb >= nblocks) return;
  const int n = (int)(a.cols - c0 < CPT ? a.cols - c0 : CPT);
  const int64_t r0 = rb * BLOCK;
  const int rows = (int)(a.rows - r0 < BLOCK ? a.rows - r0 : BLOCK);
  const unsigned char* p = static_cast<const unsigned char*>(a.X) + (r0 * a.ldx + c0) * kBytes<DT>;
  const int64_t step = a.ldx * kBytes<DT>;
  Cols<DT, CPT> v[BLOCK];
#pragma unroll
  for (int i = 0; i < BLOCK; ++i) {
    if (i < rows) {
      v[i] = load_cols<DT, CPT>(p + i * step, n);
    } else {
#pragma unroll
      for (int j = 0; j < Cols<DT, CPT>::W; ++j) v[i].w[j] = 0u;
    }
  }
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (j >= n) break;
    // The column's magnitudes; with 16-bit types the word's other column
    // is maximised along and dropped.
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < BLOCK; ++i) {
      if constexpr (DT == GEMM_DTYPE_F32) m = umax(m, v[i].w[j] & 0x7fffffffu);
      else m = pk_umax(m, v[i].w[j / 2] & 0x7fff7fffu);
    }
    if constexpr (DT != GEMM_DTYPE_F32) m = widen_bits<DT>(j % 2 ? m >> 16 : m & 0xffffu);
    const unsigned s = scale_byte<FMT>(m);
    const float factor = scale_float(s);
    constexpr int QW = kBlockBytes<FMT> / 4;
    unsigned q[QW];
#pragma unroll
    for (int w = 0; w < QW; ++w) q[w] = 0u;
    // Rows 2t, 2t+1 of column j.
    auto pair16 = [&](int t) __attribute__((always_inline)) {
      const unsigned lo = v[2 * t].w[j / 2], hi = v[2 * t + 1].w[j / 2];
      return __builtin_amdgcn_perm(hi, lo, j % 2 ? 0x07060302u : 0x05040100u);
    };
    auto put = [&](int w, int t, auto S) __attribute__((always_inline)) {
      constexpr int sel = decltype(S)::value;
      if constexpr (DT == GEMM_DTYPE_F32)
        q[w] = encode2<FMT, sel>(q[w], __builtin_bit_cast(float, v[2 * t].w[j]),
                                 __builtin_bit_cast(float, v[2 * t + 1].w[j]), factor);
      else
        q[w] = encode2<FMT, DT, sel>(q[w], pair16(t), factor);
    };
#pragma unroll
    for (int w = 0; w < QW; ++w) {
      if constexpr (FMT == GEMM_MX_E2M1) {
        put(w, 4 * w, std::integral_constant<int, 0>{});
        put(w, 4 * w + 1, std::integral_constant<int, 1>{});
        put(w, 4 * w + 2, std::integral_constant<int, 2>{});
        put(w, 4 * w + 3, std::integral_constant<int, 3>{});
      } else {
        put(w, 2 * w, std::integral_constant<int, 0>{});
        put(w, 2 * w + 1, std::integral_constant<int, 1>{});
      }
    }
    if (s == 255u)
#pragma unroll
      for (int w = 0; w < QW; ++w) q[w] = 0u;
    uint8_t* dst = a.codes + (c0 + j) * a.ldq + rb * kBlockBytes<FMT>;
#pragma unroll
    for (int w = 0; w < QW; w += 4)
      *reinterpret_cast<u32x4*>(dst + 4 * w) = u32x4{q[w], q[w + 1], q[w + 2], q[w + 3]};
    a.scales[(c0 + j) * a.lds + rb] = (uint8_t)s;
  }
}

// Two values of a code word: byte SEL (E2M1) or half-word SEL (E4M3).
template <int FMT, int SEL>
__device__ __forceinline__ f32x2 decode2(unsigned w, float factor) {
  if constexpr (FMT == GEMM_MX_E2M1)
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, factor, SEL);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, factor, SEL != 0);
}

// The same as a packed pair of a 16-bit type, rounded to nearest even.
template <int FMT, int DT, int SEL>
__device__ __forceinline__ unsigned decode2_16(unsigned w, float factor) {
  if constexpr (DT == GEMM_DTYPE_BF16) {
    if constexpr (FMT == GEMM_MX_E2M1)
      return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, factor, SEL));
    else
      return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, factor, SEL != 0));
  } else {
    const f32x2 v = decode2<FMT, SEL>(w, factor);
    return __builtin_bit_cast(unsigned, f16x2{(_Float16)v[0], (_Float16)v[1]});
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(unsigned char* row, int64_t c, int64_t n, const Eight<DT>& v) {
  unsigned char* p = row + c * kBytes<DT>;
  if (VEC && n >= 8) {
#pragma unroll
    for (int i = 0; i < Eight<DT>::W / 4; ++i)
      *reinterpret_cast<u32x4*>(p + 16 * i) = u32x4{v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]};
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= n) break;
    if constexpr (DT == GEMM_DTYPE_F32) reinterpret_cast<unsigned*>(p)[i] = v.w[i];
    else reinterpret_cast<unsigned short*>(p)[i] = (unsigned short)(v.w[i / 2] >> (16 * (i % 2)));
  }
}

template <int DT, int FMT, bool VEC, int UNROLL>
__global__ void __launch_bounds__(kThreads)
dequantize_rows(DequantArgs a, int chunks, int width_log2, int tiles_x) {
  constexpr int QB = kBlockBytes<FMT> / 4;
  const int width = 1 << width_log2;
  const int tid = threadIdx.x;
  const int ty = blockIdx.x / tiles_x, tx = blockIdx.x - ty * tiles_x;
  const int64_t row = ((int64_t)ty << (8 - width_log2)) + (tid >> width_log2);
  if (row >= a.rows) return;
  unsigned char* x = static_cast<unsigned char*>(a.X) + row * a.ldx * kBytes<DT>;
  const int64_t c0 = (int64_t)tx * width * UNROLL + (tid & (width - 1));
  unsigned q[UNROLL][2], s[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int64_t chunk = c0 + (int64_t)u * width;
    q[u][0] = q[u][1] = s[u] = 0u;
    if (chunk < chunks) {
      const uint8_t* src = a.q.codes + row * a.q.ldq + chunk * QB;
      if constexpr (FMT == GEMM_MX_E2M1) {
        q[u][0] = *reinterpret_cast<const unsigned*>(src);
      } else {
        const u32x2 t = *reinterpret_cast<const u32x2*>(src);
        q[u][0] = t[0];
        q[u][1] = t[1];
      }
      s[u] = a.q.scales[row * a.q.lds + chunk / 4];
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const int64_t chunk = c0 + (int64_t)u * width;
    if (chunk >= chunks) break;
    const float factor = scale_float(s[u]);
    Eight<DT> v;
    auto put = [&](auto I, unsigned w, auto S) __attribute__((always_inline)) {
      constexpr int i = decltype(I)::value, sel = decltype(S)::value;
      if constexpr (DT == GEMM_DTYPE_F32) {
        const f32x2 t = decode2<FMT, sel>(w, factor);
        v.w[2 * i] = __builtin_bit_cast(unsigned, (float)t[0]);
        v.w[2 * i + 1] = __builtin_bit_cast(unsigned, (float)t[1]);
      } else {
        v.w[i] = decode2_16<FMT, DT, sel>(w, factor);
      }
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 3> I3;
    if constexpr (FMT == GEMM_MX_E2M1) {
      put(I0{}, q[u][0], I0{}); put(I1{}, q[u][0], I1{}); put(I2{}, q[u][0], I2{}); put(I3{}, q[u][0], I3{});
    } else {
      put(I0{}, q[u][0], I0{}); put(I1{}, q[u][0], I1{}); put(I2{}, q[u][1], I0{}); put(I3{}, q[u][1], I1{});
    }
    store8<DT, VEC>(x, 8 * chunk, a.cols - 8 * chunk, v);
  }
}

// Transposed: the lane layout of quantize_cols, read and write exchanged.
template <int DT, int FMT, bool VEC, int RB>
__global__ void __launch_bounds__(kThreads)
dequantize_cols(DequantArgs a, int nblocks, int tiles_x) {
  constexpr int CPT = VEC ? 16 / kBytes<DT> : 1;
  constexpr int CG = 64 / RB;
  constexpr int QW = kBlockBytes<FMT> / 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ty = blockIdx.x / tiles_x, tx = blockIdx.x - ty * tiles_x;
  const int64_t c0 = ((int64_t)tx * 4 + wave) * (CG * CPT) + (lane / RB) * CPT;
  const int64_t rb = (int64_t)ty * RB + lane % RB;
  if (c0 >= a.cols || rb >= nblocks) return;
  const int n = (int)(a.cols - c0 < CPT ? a.cols - c0 : CPT);
  const int64_t r0 = rb * BLOCK;
  const int rows = (int)(a.rows - r0 < BLOCK ? a.rows - r0 : BLOCK);
  unsigned q[CPT][QW];
  float factor[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int64_t c = c0 + (j < n ? j : 0);  // columns past the last repeat the first and are not stored
    const uint8_t* src = a.q.codes + c * a.q.ldq + rb * kBlockBytes<FMT>;
#pragma unroll
    for (int w = 0; w < QW; w += 4) {
      const u32x4 t = *reinterpret_cast<const u32x4*>(src + 4 * w);
#pragma unroll
      for (int k = 0; k < 4; ++k) q[j][w + k] = t[k];
    }
    factor[j] = scale_float(a.q.scales[c * a.q.lds + rb]);
  }
  unsigned char* p = static_cast<unsigned char*>(a.X) + (r0 * a.ldx + c0) * kBytes<DT>;
  const int64_t step = a.ldx * kBytes<DT>;
  // Rows 2t, 2t+1.
  auto two_rows = [&](int t, unsigned (*w_of)[QW], auto S) __attribute__((always_inline)) {
    constexpr int sel = decltype(S)::value;
    constexpr int PER = FMT == GEMM_MX_E2M1 ? 4 : 2;  // pairs per code word
    const int w = t / PER;
    Cols<DT, CPT> lo, hi;
    if constexpr (DT == GEMM_DTYPE_F32) {
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const f32x2 v = decode2<FMT, sel>(w_of[j][w], factor[j]);
        lo.w[j] = __builtin_bit_cast(unsigned, (float)v[0]);
        hi.w[j] = __builtin_bit_cast(unsigned, (float)v[1]);
      }
    } else if constexpr (CPT == 1) {
      const unsigned v = decode2_16<FMT, DT, sel>(w_of[0][w], factor[0]);
      lo.w[0] = v & 0xffffu;
      hi.w[0] = v >> 16;
    } else {
#pragma unroll
      for (int j = 0; j < CPT; j += 2) {
        const unsigned x = decode2_16<FMT, DT, sel>(w_of[j][w], factor[j]);
        const unsigned y = decode2_16<FMT, DT, sel>(w_of[j + 1][w], factor[j + 1]);
        lo.w[j / 2] = __builtin_amdgcn_perm(y, x, 0x05040100u);
        hi.w[j / 2] = __builtin_amdgcn_perm(y, x, 0x07060302u);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * t + h >= rows) break;
      const Cols<DT, CPT>& v = h ? hi : lo;
      unsigned char* d = p + (2 * t + h) * step;
      bool done = false;
      if constexpr (CPT > 1) {
        if (n >= CPT) {
          *reinterpret_cast<u32x4*>(d) = u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
          done = true;
        }
      }
      if (!done) {
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          if (j >= n) break;
          if constexpr (DT == GEMM_DTYPE_F32) reinterpret_cast<unsigned*>(d)[j] = v.w[j];
          else reinterpret_cast<unsigned short*>(d)[j] = (unsigned short)(v.w[j / 2] >> (16 * (j % 2)));
        }
      }
    }
  };
#pragma unroll
  for (int t = 0; t < BLOCK / 2; ++t) {
    constexpr int PER = FMT == GEMM_MX_E2M1 ? 4 : 2;
    switch (t % PER) {
      case 0: two_rows(t, q, std::integral_constant<int, 0>{}); break;
      case 1: two_rows(t, q, std::integral_constant<int, 1>{}); break;
      case 2: two_rows(t, q, std::integral_constant<int, FMT == GEMM_MX_E2M1 ? 2 : 0>{}); break;
      default: two_rows(t, q, std::integral_constant<int, FMT == GEMM_MX_E2M1 ? 3 : 1>{}); break;
    }
  }
}

// Grid of the row kernels: lanes across a row (a power of two of at least a
// block's four) and workgroups along a row.
struct RowGrid {
  int width_log2, tiles_x;
};
RowGrid row_grid(int chunks, int unroll) {
  RowGrid g;
  g.width_log2 = 2;
  while (g.width_log2 < 8 && (1 << g.width_log2) < chunks) ++g.width_log2;
  const int per = (1 << g.width_log2) * unroll;
  g.tiles_x = (chunks + per - 1) / per;
  return g;
}

// Chunks a lane holds along a row: enough bytes in flight to cover the
// memory latency once there are waves for every CU; one where there are few.
constexpr int kUnroll = 4;
bool unrolled(int rows, int chunks) { return (int64_t)rows * chunks >= (int64_t)256 * 1024 * kUnroll; }

template <class F>
hipError_t by_types(int dtype, int format, F&& f) {
  typedef std::integral_constant<int, GEMM_MX_E2M1> Q4;
  typedef std::integral_constant<int, GEMM_MX_E4M3> Q8;
  typedef std::integral_constant<int, GEMM_DTYPE_F32> TF;
  typedef std::integral_constant<int, GEMM_DTYPE_F16> TH;
  typedef std::integral_constant<int, GEMM_DTYPE_BF16> TB;
  auto with = [&](auto DT) { return format == GEMM_MX_E2M1 ? f(DT, Q4{}) : f(DT, Q8{}); };
  return dtype == GEMM_DTYPE_F32 ? with(TF{}) : dtype == GEMM_DTYPE_F16 ? with(TH{}) : with(TB{});
}

// 16-byte accesses to X's rows.
template <int DT>
bool vector_rows(const void* X, int64_t ldx) {
  return ((uintptr_t)X & 15) == 0 && (ldx * kBytes<DT>) % 16 == 0;
}

// Workgroups of one launch: a grid holds fewer than 2^32 work-items, so
// taller matrices go in slices of rows.
constexpr int64_t kMaxGroups = 1 << 22;

// launch(grid, row grid, first row, rows) over slices along the rows.
template <class F>
hipError_t slice_rows(int rows, int chunks, int unroll, F&& launch) {
  const RowGrid g = row_grid(chunks, unroll);
  const int64_t rpg = kThreads >> g.width_log2;
  const int64_t per = kMaxGroups / g.tiles_x * rpg;  // tiles_x < 2^19
  for (int64_t r0 = 0; r0 < rows; r0 += per) {
    const int64_t n = rows - r0 < per ? rows - r0 : per;
    const hipError_t e = launch(dim3((unsigned)((n + rpg - 1) / rpg * g.tiles_x)), g, r0, (int)n);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// launch(grid, tiles along a row, first row, rows) over slices of whole
// groups of rb row blocks.
template <class F>
hipError_t slice_cols(int rows, int cols, int64_t span, int rb, F&& launch) {
  const int64_t tiles_x = (cols + span - 1) / span;  // < 2^24
  const int64_t step = (int64_t)rb * BLOCK;
  const int64_t fit = kMaxGroups / tiles_x;
  const int64_t per = (fit < 1 ? 1 : fit) * step;
  for (int64_t r0 = 0; r0 < rows; r0 += per) {
    const int64_t n = rows - r0 < per ? rows - r0 : per;
    const hipError_t e = launch(dim3((unsigned)((n + step - 1) / step * tiles_x)), (int)tiles_x, r0, (int)n);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize(int dtype, int format, bool trans, const QuantArgs& args, hipStream_t stream) {
  if (args.rows <= 0 || args.cols <= 0) return hipSuccess;
  return by_types(dtype, format, [&](auto DT_, auto FMT_) {
    constexpr int DT = decltype(DT_)::value, FMT = decltype(FMT_)::value;
    const bool vec = vector_rows<DT>(args.X, args.ldx);
    const dim3 block(kThreads);
    QuantArgs a = args;
    if (!trans) {
      const int chunks = (int)(4 * blocks_of(a.cols));
      const bool many = unrolled(a.rows, chunks);
      return slice_rows(args.rows, chunks, many ? kUnroll : 1, [&](dim3 grid, const RowGrid& g, int64_t r0, int n) {
        a.X = static_cast<const unsigned char*>(args.X) + r0 * a.ldx * kBytes<DT>;
        a.codes = args.codes + r0 * a.ldq;
        a.scales = args.scales + r0 * a.lds;
        a.rows = n;
        if (vec && many)
          hipLaunchKernelGGL((quantize_rows<DT, FMT, true, kUnroll>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        else if (vec)
          hipLaunchKernelGGL((quantize_rows<DT, FMT, true, 1>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        else if (many)
          hipLaunchKernelGGL((quantize_rows<DT, FMT, false, kUnroll>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        else
          hipLaunchKernelGGL((quantize_rows<DT, FMT, false, 1>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        return hipGetLastError();
      });
    }
    const int rb = vec ? 4 : 1;
    const int64_t span = 4 * (int64_t)(64 / rb) * (vec ? 16 / kBytes<DT> : 1);
    return slice_cols(args.rows, args.cols, span, rb, [&](dim3 grid, int tiles_x, int64_t r0, int n) {
      a.X = static_cast<const unsigned char*>(args.X) + r0 * a.ldx * kBytes<DT>;
      a.codes = args.codes + r0 / BLOCK * kBlockBytes<FMT>;
      a.scales = args.scales + r0 / BLOCK;
      a.rows = n;
      const int nblocks = (n + BLOCK - 1) / BLOCK;
      if (vec)
        hipLaunchKernelGGL((quantize_cols<DT, FMT, true, 4>), grid, block, 0, stream, a, nblocks, tiles_x);
      else
        hipLaunchKernelGGL((quantize_cols<DT, FMT, false, 1>), grid, block, 0, stream, a, nblocks, tiles_x);
      return hipGetLastError();
    });
  });
}

hipError_t launch_dequantize(int dtype, int format, bool trans, const DequantArgs& args, hipStream_t stream) {
  if (args.rows <= 0 || args.cols <= 0) return hipSuccess;
  return by_types(dtype, format, [&](auto DT_, auto FMT_) {
    constexpr int DT = decltype(DT_)::value, FMT = decltype(FMT_)::value;
    const bool vec = vector_rows<DT>(args.X, args.ldx);
    const dim3 block(kThreads);
    DequantArgs a = args;
    if (!trans) {
      const int chunks = (int)ceil_div(a.cols, 8);
      const bool many = unrolled(a.rows, chunks);
      return slice_rows(args.rows, chunks, many ? kUnroll : 1, [&](dim3 grid, const RowGrid& g, int64_t r0, int n) {
        a.X = static_cast<unsigned char*>(args.X) + r0 * a.ldx * kBytes<DT>;
        a.q.codes = args.q.codes + r0 * a.q.ldq;
        a.q.scales = args.q.scales + r0 * a.q.lds;
        a.rows = n;
        if (vec && many)
          hipLaunchKernelGGL((dequantize_rows<DT, FMT, true, kUnroll>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        else if (vec)
          hipLaunchKernelGGL((dequantize_rows<DT, FMT, true, 1>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        else if (many)
          hipLaunchKernelGGL((dequantize_rows<DT, FMT, false, kUnroll>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        else
          hipLaunchKernelGGL((dequantize_rows<DT, FMT, false, 1>), grid, block, 0, stream, a, chunks, g.width_log2, g.tiles_x);
        return hipGetLastError();
      });
    }
    const int rb = vec ? 4 : 1;
    const int64_t span = 4 * (int64_t)(64 / rb) * (vec ? 16 / kBytes<DT> : 1);
    return slice_cols(args.rows, args.cols, span, rb, [&](dim3 grid, int tiles_x, int64_t r0, int n) {
      a.X = static_cast<unsigned char*>(args.X) + r0 * a.ldx * kBytes<DT>;
      a.q.codes = args.q.codes + r0 / BLOCK * kBlockBytes<FMT>;
      a.q.scales = args.q.scales + r0 / BLOCK;
      a.rows = n;
      const int nblocks = (n + BLOCK - 1) / BLOCK;
      if (vec)
        hipLaunchKernelGGL((dequantize_cols<DT, FMT, true, 4>), grid, block, 0, stream, a, nblocks, tiles_x);
      else
        hipLaunchKernelGGL((dequantize_cols<DT, FMT, false, 1>), grid, block, 0, stream, a, nblocks, tiles_x);
      return hipGetLastError();
    });
  });
}

}  // namespace mx
}  // namespace gemm

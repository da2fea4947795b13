// Building blocks of the pipelined microscaled products (mx_matmul.hip,
// mx_wgrad.hip): LDS-direct copies through buffer descriptors, the K loop's
// barrier, matrix instructions with accumulators tied in place, and the
// register transposition before 16-bit stores.
#pragma once

#include <utility>

#include "mx_bounds.h"
#include "mx_internal.h"

namespace gemm {
namespace mx {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef __attribute__((address_space(3))) unsigned lds_u32;

template <int I>
using IC = std::integral_constant<int, I>;

template <class F, int... I>
__device__ __forceinline__ void static_for(F&& f, std::integer_sequence<int, I...>) {
  (f(IC<I>{}), ...);
}

// A raw buffer over [base, base + bytes), at most 2^31 - 1 of them: loads
// past its end give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int64_t n = bytes < 0 ? 0 : bytes > 0x7fffffff ? 0x7fffffff : bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)n, 0x00020000);
}

// Barrier of the K loop: this wave's LDS reads have returned and its copies
// landed; no memory fence beyond that (the loop's LDS traffic is those).
__device__ __forceinline__ void loop_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The matrix instructions as inline assembly, their accumulators tied in
// place: with the builtins the register allocator moves the four-register
// accumulators of a 128 x 128 wave tile about on every pass.  The compiler's
// hazard checks do not see into the assembly, so the kernels keep other
// writers of an operand at least 4 wait states before its reader (operands
// come from LDS reads, or are decoded several instructions ahead), and
// touch the accumulators only outside a guard.
// (BYTE: the byte of both scale operands that counts.)
template <int BYTE>
__device__ __forceinline__ void mfma_fp4_asm(f32x4& c, i32x4 a, i32x4 b, int sa, int sb) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (BYTE == 0)
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  else
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                 : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
#endif
}
__device__ __forceinline__ void mfma_bf16_asm(f32x4& c, i32x4 a, i32x4 b) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
#endif
}

// 24 wait states with nothing scheduled across: more than any matrix-core
// hazard of gfx950 needs.
__device__ __forceinline__ void mfma_guard() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The accumulators as values known in their registers at this point: what
// precedes it wrote them, what follows reads them.  A guard alone is no
// fence for them (the compiler read results ahead of it).
template <int NB, int MB>
__device__ __forceinline__ void pin(f32x4 (&acc)[NB][MB]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i) asm volatile("" : "+a"(acc[j][i]));
#endif
}

// Eight codes (tokens in order) of one block -> eight bfloat16 values.
__device__ __forceinline__ u32x4 decode8(u32x2 w, float factor) {
  u32x4 v;
  v[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], factor, false));
  v[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], factor, true));
  v[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], factor, false));
  v[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], factor, true));
  return v;
}

// Stores of one 16-row block row of a wave's tile, through a buffer over C
// (so without branches: what lies outside the matrix gets an offset past
// the range).  Block nb's register i of lane l is element (l%16, 16nb +
// 4(l/16) + i) of the tile; `row` is the byte offset of the lane's row (OOB:
// none), `cols` of the tile's columns are inside the matrix.
//  * FP32: a lane's four values are one 16-byte store, four lanes 64 bytes.
//  * 16 bits: blocks nb and nb + 1 exchange odd and even 16-lane rows
//    (v_permlane16_swap), which leaves lane row q with columns 8(q/2) .. +7
//    of block nb + q%2: again 16-byte stores, four lanes 64 bytes.
// VEC: rows are 16-byte aligned and a whole number of 16-byte groups long;
// otherwise element by element.
template <int DT, int NB, bool VEC>
__device__ __forceinline__ void store_block_row(const void* C, unsigned row, int cols, const f32x4 (&v)[NB], int q) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename TypeOf<DT>::type T;
  constexpr unsigned es = sizeof(T);
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(C, 0x7fffffff);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int n = 16 * nb + 4 * q;
      if constexpr (VEC) {
        const unsigned off = n < cols ? row + n * es : OOB;
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v[nb]), rc, off, 0, 2);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = v[nb][i];  // (a vector's element bit-cast in place is its first)
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), rc,
                                                n + i < cols ? row + (n + i) * es : OOB, 0, 0);
        }
      }
    }
  } else {
    typedef T t2 __attribute__((ext_vector_type(2)));
    static_assert(NB % 2 == 0, "blocks in pairs");
#pragma unroll
    for (int nb = 0; nb < NB; nb += 2) {
      unsigned x[2], y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = __builtin_bit_cast(unsigned, t2{(T)v[nb][2 * i], (T)v[nb][2 * i + 1]});
        y[i] = __builtin_bit_cast(unsigned, t2{(T)v[nb + 1][2 * i], (T)v[nb + 1][2 * i + 1]});
      }
      const u32x2 s0 = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false));
      const u32x2 s1 = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false));
      const u32x4 w = {s0[0], s1[0], s0[1], s1[1]};
      const int n = 16 * (nb + q % 2) + 8 * (q / 2);
      if constexpr (VEC) {
        const unsigned off = n < cols ? row + n * es : OOB;
        __builtin_amdgcn_raw_buffer_store_b128(w, rc, off, 0, 2);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(w[i / 2] >> (16 * (i % 2))), rc,
                                                n + i < cols ? row + (n + i) * es : OOB, 0, 0);
      }
    }
  }
#endif
}

// The old values of the same block row (zeros outside), in the accumulators'
// layout.  Branch-free like the stores: divergent branches between the
// accumulators' uses make the register allocator move them about under a
// partial execution mask.
template <int DT, int NB, bool VEC>
__device__ __forceinline__ void load_block_row(const void* C, unsigned row, int cols, f32x4 (&v)[NB], int q) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename TypeOf<DT>::type T;
  constexpr unsigned es = sizeof(T);
  const __amdgpu_buffer_rsrc_t rc = make_rsrc(C, 0x7fffffff);
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int n = 16 * nb + 4 * q;
    if constexpr (VEC && es == 4) {
      v[nb] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rc, n < cols ? row + n * es : OOB, 0, 0));
    } else if constexpr (VEC) {
      typedef T t4 __attribute__((ext_vector_type(4)));
      const t4 t = __builtin_bit_cast(t4, __builtin_amdgcn_raw_buffer_load_b64(rc, n < cols ? row + n * es : OOB, 0, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[nb][i] = (float)t[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned off = n + i < cols ? row + (n + i) * es : OOB;
        if constexpr (es == 4)
          v[nb][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rc, off, 0, 0));
        else
          v[nb][i] = (float)__builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(rc, off, 0, 0));
      }
    }
  }
#endif
}

}  // namespace mx
}  // namespace gemm

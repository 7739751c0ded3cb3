// Device helpers of the dense operators (kernels_dense.hip, kernels_w4.hip): 16-bit elements
// of either type, their MFMA forms, and the gated block's activations.  gfx950 only.
#pragma once

#include "device_common.h"

namespace ft {
namespace dev {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ---- 16-bit elements (H: fp16, else bf16) -----------------------------------------

template <bool H>
__device__ __forceinline__ f32x16_t mfma32(i32x4_t a, i32x4_t b, f32x16_t c) {
  if constexpr (H)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
template <bool H>
__device__ __forceinline__ f32x4_t mfma16(i32x4_t a, i32x4_t b, f32x4_t c) {
  if constexpr (H)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
// Two fp32 values to one word of two elements, nearest even, the first in the low half.
template <bool H>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (H) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)lo, (_Float16)hi});
  } else {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, b2{(__bf16)lo, (__bf16)hi});
  }
}
template <bool H>
__device__ __forceinline__ float lo16(uint32_t w) {
  if constexpr (H) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return (float)__builtin_bit_cast(h2, w).x;
  } else {
    return bf_lo(w);
  }
}
template <bool H>
__device__ __forceinline__ float hi16(uint32_t w) {
  if constexpr (H) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return (float)__builtin_bit_cast(h2, w).y;
  } else {
    return bf_hi(w);
  }
}
template <bool H>
__device__ __forceinline__ float to_f32(uint16_t v) {
  return lo16<H>(v);
}

// A buffer without an end of its own: offsets are checked against kOOB alone.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p) { return buf_rsrc(p, 0x7fffffffu); }

__device__ __forceinline__ uint2 buf_ld8b(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  typedef int i32x2_t __attribute__((ext_vector_type(2)));
  const i32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
  return make_uint2((uint32_t)v.x, (uint32_t)v.y);
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)p);
}

// Quads q = 2j and 2j + 1 of a 32x32 result (4 consecutive n each, in two words of two 16-bit
// elements) exchanged between lanes l and l + 32: lane l < 32 gets n = 16j .. 16j + 7, lane
// l + 32 gets 16j + 8 .. 16j + 15.  Its own inverse.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const u32x2_t r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r.x;
  b = r.y;
}

// ---- activations --------------------------------------------------------------------
// act(z) and act'(z).  Every value that leaves these is rounded to 16 bits (or 8) after, so
// exp and the reciprocal are the hardware's (a few ulp of fp32).

struct ActD {
  float f, df;
};
__device__ __forceinline__ float act_f(float z, int act) {
  if (act == FT_ACT_SILU) return silu_fast(z);
  // gelu, tanh form: z/2 (1 + tanh w) = z / (1 + e^-2w), w = sqrt(2/pi) (z + 0.044715 z^3)
  const float w2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
  return z * __builtin_amdgcn_rcpf(1.0f + __expf(-w2));
}
__device__ __forceinline__ ActD act_df(float z, int act) {
  ActD r;
  if (act == FT_ACT_SILU) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    r.f = z * s;
    r.df = s * (1.0f + z * (1.0f - s));
  } else {
    // with s = 1/(1 + e^-2w): f = z s, f' = s + z s (1 - s) (2w)'
    // (past |z| = 10^5 s is 0 or 1 and s (1 - s) is 0: a square past fp32 would make that NaN)
    const float zz = fminf(z * z, 1e10f);
    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-1.5957691216057308f * (z + 0.044715f * z * zz)));
    r.f = z * s;
    r.df = s + z * (s * (1.0f - s)) * (1.5957691216057308f * (1.0f + 0.134145f * zz));
  }
  return r;
}

}  // namespace dev
}  // namespace ft

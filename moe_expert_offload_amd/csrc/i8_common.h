// Device helpers of the products in 8-bit integers (kernels_i8.hip, kernels_moe.hip): a row's scale
// and its codes, and the integer MFMA forms.  gfx950 only.
#pragma once

#include "dense_common.h"

namespace ft {
namespace dev {

typedef int i32x16_t __attribute__((ext_vector_type(16)));

// Sums of products of 8-bit integers, exact in 32 bits: lane l supplies 16 consecutive bytes of k of
// row l % 32 (l % 16), both operands alike; results lie as those of the 16-bit forms do.
__device__ __forceinline__ i32x16_t mfma32(i32x4_t a, i32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ i32x4_t mfma16(i32x4_t a, i32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// ---- a row in 8 bits: scale s = max|x| / 127 in fp32, code = x / s to nearest, ties to even -------
// Codes are those of the exact quotient.  x is a 16-bit float and s an fp32 number, so near the
// borders between codes, (q + 1/2) s, the remainder x - q s is a multiple of s's last place below 2 s:
// one fma gives it exactly.  q comes from a product with 1 / s, which is off by at most one next to
// a border, and is corrected where the remainder passes s / 2.
struct RowScale {
  float scale;            // as stored: NaN for a row that is not finite, 0 for a row of zeros
  float s, inv, half, up;  // s and x times `up`, which lifts tiny rows out of the subnormals
  bool finite;
};
// amax: the largest magnitude's 16 bits, as a whole number (infinities and NaN order above the rest).
template <bool H>
__device__ __forceinline__ RowScale row_scale(uint32_t amax) {
  RowScale r;
  r.finite = amax < (H ? 0x7c00u : 0x7f80u);
  const float top = to_f32<H>((uint16_t)amax);
  r.scale = r.finite ? top / 127.0f : __uint_as_float(0x7fc00000u);
  r.up = top < 0x1p-60f ? 0x1p64f : 1.0f;
  r.s = r.finite ? r.scale * r.up : 0.0f;
  r.inv = r.s > 0.0f ? 1.0f / r.s : 0.0f;
  r.half = r.s > 0.0f ? 0.5f * r.s : 1.0f;
  return r;
}
// 8 elements (4 words) to 8 codes.
template <bool H>
__device__ __forceinline__ uint2 row_codes8(const uint32_t (&w)[4], const RowScale& r) {
  float x[8], q[8], rem[8], far = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = (e & 1 ? hi16<H>(w[e >> 1]) : lo16<H>(w[e >> 1])) * r.up;
    q[e] = rintf(x[e] * r.inv);
    rem[e] = fmaf(-q[e], r.s, x[e]);
    far = fmaxf(far, fabsf(rem[e]));
  }
  if (far >= r.half) {  // next to a border: seldom
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float odd = fabsf(q[e] - 2.0f * truncf(0.5f * q[e]));  // 1 for odd q
      if (rem[e] > r.half || (rem[e] == r.half && odd != 0.0f))
        q[e] += 1.0f;
      else if (rem[e] < -r.half || (rem[e] == -r.half && odd != 0.0f))
        q[e] -= 1.0f;
    }
  }
  uint32_t v[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = (uint32_t)(int)q[4 * h + e];
    // bytes 0 of the four, in order
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
    v[h] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  }
  return r.finite ? make_uint2(v[0], v[1]) : make_uint2(0, 0);
}
// The larger of two words of two magnitudes each, half by half, into one.
__device__ __forceinline__ uint32_t amax_of(uint32_t w, uint32_t m) {
  const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu, t = a > b ? a : b;
  return t > m ? t : m;
}
__device__ __forceinline__ uint32_t amax4(const uint4& v, uint32_t m) {
  return amax_of(v.w, amax_of(v.z, amax_of(v.y, amax_of(v.x, m))));
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t w = (uint32_t)__shfl_xor((int)v, o, WAVE);
    v = w > v ? w : v;
  }
  return v;
}

// One row of n elements to codes and its scale by ROWT threads, 64 or a whole block (`red`: a word of LDS for each wave). The row is
// held in registers between its largest element and its codes, NP pieces of 8 elements a thread; what is
// longer is read again.  place(i): where the codes of 8 elements from 8 i go (a uint2).
template <bool H, int ROWT, int NP, class Place>
__device__ __forceinline__ void quant_row(const uint16_t* src, int n, Place place, float* scale, uint32_t* red) {
  const int at = threadIdx.x % ROWT, pieces = n >> 3;
  const uint4* q = reinterpret_cast<const uint4*>(src);
  uint4 v[NP];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) v[i] = at + i * ROWT < pieces ? q[at + i * ROWT] : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < NP; ++i) m = amax4(v[i], m);
  for (int p = at + NP * ROWT; p < pieces; p += ROWT) m = amax4(q[p], m);
  m = wave_umax(m);
  if constexpr (ROWT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < ROWT / 64; ++w) m = max(m, red[w]);
  }
  const RowScale r = row_scale<H>(m);
  auto put = [&](int p, const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    *place(p) = row_codes8<H>(w, r);
  };
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (at + i * ROWT < pieces) put(at + i * ROWT, v[i]);
  for (int p = at + NP * ROWT; p < pieces; p += ROWT) put(p, q[p]);
  if (at == 0) *scale = r.scale;
}
// One after another; codes may lie in LDS.
template <bool H, int ROWT, int NP>
__device__ __forceinline__ void quant_row(const uint16_t* src, int n, int8_t* codes, float* scale, uint32_t* red) {
  uint2* d = reinterpret_cast<uint2*>(codes);
  quant_row<H, ROWT, NP>(src, n, [=](int i) { return d + i; }, scale, red);
}

// A product's value: the whole-number sum times the channel's scale, then the token's.
__device__ __forceinline__ float i8_value(int acc, float channel, float token) { return ((float)acc * channel) * token; }

}  // namespace dev
}  // namespace ft

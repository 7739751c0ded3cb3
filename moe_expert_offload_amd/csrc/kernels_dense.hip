// Dense operators beside the grouped experts: the gated feed-forward block (forward and
// backward), and activations kept in 8 bits.  gfx950 only.
//
//   a = x Wg^T, u = x Wu^T, h = act(a) * u, y = h Wd^T (+ residual)
//   dh = dy Wd, du = dh act(a), da = dh u act'(a)
//   dWd = dy^T h, dWg = da^T x, dWu = du^T x, dx = da Wg + du Wu
//
// h, da and du are rounded to the activations' type as they leave their product's epilogue, because they
// are the operands of the next 16-bit MFMA: keeping them in fp32 would take two or three products (high and low
// parts) for one. Together with the result's rounding that is 1.4 times the error of fp32 rounded once (bf16
// 2.3e-3 against 1.7e-3, fp16 2.9e-4 against 2.1e-4, over the elements' rms). Everything else is fp32.
#include <type_traits>

#include "dense_common.h"
#include "dense_cut.h"

namespace ft {

using namespace dev;

namespace {

// ---- MX8: 32 values under one power of two, E4M3 codes ------------------------------

// The scale byte of a block whose largest finite magnitude is amax: e + 127 for the least
// e >= -127 with amax <= 448 * 2^e, so no code saturates and each is within half a step
// (2^-4 relative).  From the bits: amax = m * 2^p with m in [1, 2) needs e = p - 8 when
// m <= 1.75, else p - 7.
__device__ __forceinline__ int mx8_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u);  // biased by 127; fp32 subnormals give <= 0
  return e < 0 ? 0 : e;
}
__device__ __forceinline__ bool finite32(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
// Four values to four codes; a value that is not finite becomes the NaN code.
__device__ __forceinline__ uint32_t mx8_codes4(float v0, float v1, float v2, float v3, int sc) {
  const int k = 127 - sc;
  const float nan = __uint_as_float(0x7fc00000u);
  const float w0 = finite32(v0) ? ldexpf(v0, k) : nan, w1 = finite32(v1) ? ldexpf(v1, k) : nan;
  const float w2 = finite32(v2) ? ldexpf(v2, k) : nan, w3 = finite32(v3) ? ldexpf(v3, k) : nan;
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(w0, w1, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(w2, w3, r, true);
}
__device__ __forceinline__ float fin_abs(float v) { return finite32(v) ? fabsf(v) : 0.0f; }
__device__ __forceinline__ void mx8_values4(uint32_t c, int sc, float* v) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  const int k = sc - 127;
  v[0] = ldexpf(a.x, k);
  v[1] = ldexpf(a.y, k);
  v[2] = ldexpf(b.x, k);
  v[3] = ldexpf(b.y, k);
  if (sc > 246) {
    // past fp32 (from 1.9375 * 2^127 on a finite value is packed to 2^128): its largest value, not an infinity,
    // whose slope would be NaN
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v[e] > 0x1.fffffep127f ? 0x1.fffffep127f : (v[e] < -0x1.fffffep127f ? -0x1.fffffep127f : v[e]);
  }
}
// A 16-bit type holds less than a code times its scale may be: its largest finite value stands for more.
template <bool H>
__device__ __forceinline__ float fit16(float v) {
  constexpr float top = H ? 65504.0f : 0x1.fep127f;
  return v > top ? top : (v < -top ? -top : v);
}

// ---- the tiled product ----------------------------------------------------------------
// C[M, N] = sum over k of A[m, k] B[n, k], each operand either row-major along k or along its
// own rows (transposed), 16-bit elements, fp32 sums on v_mfma_f32_32x32x16.
//
// A block computes a BM x BN tile with WM x WN waves of (BM / WM) x 64.  K runs in stages of
// 64: both operands go straight from memory into one of two LDS buffers, one stage ahead.
//   - An operand along k: LDS rows of 64 elements (128 bytes), the 16-byte piece p of row r at
//     place p ^ (r / 2 & 7): the 16 rows of a read phase then use all 16 pieces of two rows'
//     banks once (p ^ (r & 7) put rows r and r + 8 on the same banks: twice the LDS cycles).
//   - A transposed operand: LDS rows are the 64 k of the stage, each BM (or BN) elements,
//     piece p of row k at p ^ ((k & 3) << 2); fragments come through the transposing LDS read
//     (16 lanes read 4 rows of k and get one column of 4 k each), whose 4 rows then fall
//     into different 64-byte parts of the banks.
// The B operand (the weights, or the N side) goes into the MFMA's first operand: a lane then
// holds one row m and groups of 4 consecutive n, which pack into wide stores.

enum {
  kGateUp,  // A = x, B = 32 rows of Wg then 32 rows of Wu per wave; h, and a and u when kept
  kOut,     // C (+ residual) to 16 bits or fp32
  kDh,      // dh = dy Wd, then h, da and du from a and u; or dh itself in fp32, where a and u were not kept
  kAgain,   // as kGateUp, then h, da and du from a, u and that dh
  kDx,      // two pieces of k: da Wg + du Wu
  kDw       // A and B transposed; rows of C from `split` on go to a second matrix
};

// Modes that compute Wg and Wu side by side.
template <int MODE>
constexpr bool kBeside = MODE == kGateUp || MODE == kAgain;

struct GemmArgs {
  const uint16_t *a, *b, *b2;  // b2: Wu (kGateUp: beside b; kDx: second piece of k)
  int64_t lda, ldb;
  int M, N, K;
  int act;
  void *c, *c2;  // c2: kDw rows from `split` on
  int64_t ldc;
  int split, c_f32;
  const void* res;
  int64_t ldr;
  // kGateUp: where a and u go (null: not kept); kDh: where they come from (null: dh to c); kAgain: dh in c
  void *sa, *su;
  uint8_t *sca, *scu;  // MX8 scales, null for 16-bit a and u
  uint16_t *h, *dag;   // kDh outputs: h [M, N], da and du [M, 2N]
  int tiles_m, tiles_n;
  // gemm256_kernel: the first `whole` tiles have a block each; of the other `rest` tiles (0: none), every
  // `group` tiles' stages are one line that `blocks` blocks share in pieces of `per`; `parts` in all.
  // gemm_kernel: all tiles (rest > 0) or none are shared, one a group.
  int whole, rest, group, blocks, per, parts;
  float* part;  // sums of pieces
};

// Tile index to its place: consecutive tiles walk 8 tile rows per column of tiles.
struct TilePos {
  int m, n;
};
__device__ __forceinline__ TilePos tile_pos(const GemmArgs& p, int t) {
  const int per = 8 * p.tiles_n, grp = t / per, first = grp * 8;
  const int rows = min(8, p.tiles_m - first), in = t - grp * per;
  return {first + in % rows, in / rows};
}

// What becomes of one 32-row piece of a wave's result: c0 and c1 are its 32x32 results at columns
// nb0 and nb1 (kGateUp: a and u of the same columns).  The lane holds row m of those from mu on, and in
// quad q the columns 8 q + 4 hi + 0..3 of each.
template <int MODE, bool H>
__device__ __forceinline__ void epilogue(const GemmArgs& p, const f32x16_t& c0, const f32x16_t& c1, int mu, int m,
                                         int nb0, int nb1, int hi) {
  const bool mok = m < p.M;
  if constexpr (MODE == kGateUp) {
    const int nb = nb0;  // the 32 columns of a, u and h
    if (p.sca) {
      // whole blocks of 32 (N % 32 == 0): this lane and its other half hold one block of row m
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float am = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) am = fmaxf(am, fin_abs((j ? c1 : c0)[e]));
        am = fmaxf(am, __shfl_xor(am, 32, WAVE));
        const int sc = mx8_scale(am);
        uint8_t* cd = static_cast<uint8_t*>(j ? p.su : p.sa) + (int64_t)m * p.N + nb;
        if (mok && nb < p.N) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint32_t*>(cd + 8 * q + 4 * hi) = mx8_codes4(
                (j ? c1 : c0)[4 * q], (j ? c1 : c0)[4 * q + 1], (j ? c1 : c0)[4 * q + 2], (j ? c1 : c0)[4 * q + 3], sc);
          if (hi == 0) (j ? p.scu : p.sca)[(int64_t)m * (p.N >> 5) + (nb >> 5)] = (uint8_t)sc;
        }
      }
    } else if (p.sa) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint16_t* dst = static_cast<uint16_t*>(j ? p.su : p.sa) + (int64_t)m * p.N;
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack2<H>((j ? c1 : c0)[4 * q + 2 * e], (j ? c1 : c0)[4 * q + 2 * e + 1]);
          swap_halves(w[0], w[2]);
          swap_halves(w[1], w[3]);
          const int n = nb + 8 * q + 8 * hi;
          if (mok && n < p.N) *reinterpret_cast<uint4*>(dst + n) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 4 * q + 2 * e;
        w[e] = pack2<H>(act_f(c0[k], p.act) * c1[k], act_f(c0[k + 1], p.act) * c1[k + 1]);
      }
      swap_halves(w[0], w[2]);
      swap_halves(w[1], w[3]);
      const int n = nb + 8 * q + 8 * hi;
      if (mok && n < p.N) *reinterpret_cast<uint4*>(p.h + (int64_t)m * p.N + n) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else if constexpr (MODE == kAgain) {
    const auto rd = rsrc_of(static_cast<const float*>(p.c) + (int64_t)mu * p.N);
    float4 g[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = nb0 + 8 * q + 4 * hi;
      const uint4 v = buf_ld16(rd, mok && n < p.N ? (uint32_t)(((m - mu) * p.N + n) * 4) : kOOB);
      g[q] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    }
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      uint32_t oh[4], oa[4], ou[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 4 * q + 2 * e;
        const float4 d = g[q + (e >> 1)];
        const float d0 = e & 1 ? d.z : d.x, d1 = e & 1 ? d.w : d.y;
        const ActD f0 = act_df(c0[k], p.act), f1 = act_df(c0[k + 1], p.act);
        oh[e] = pack2<H>(f0.f * c1[k], f1.f * c1[k + 1]);
        oa[e] = pack2<H>(d0 * c1[k] * f0.df, d1 * c1[k + 1] * f1.df);
        ou[e] = pack2<H>(d0 * f0.f, d1 * f1.f);
      }
      swap_halves(oh[0], oh[2]);
      swap_halves(oh[1], oh[3]);
      swap_halves(oa[0], oa[2]);
      swap_halves(oa[1], oa[3]);
      swap_halves(ou[0], ou[2]);
      swap_halves(ou[1], ou[3]);
      const int n = nb0 + 8 * q + 8 * hi;
      if (mok && n < p.N) {
        *reinterpret_cast<uint4*>(p.h + (int64_t)m * p.N + n) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
        uint16_t* dg = p.dag + 2 * (int64_t)m * p.N + n;
        *reinterpret_cast<uint4*>(dg) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        *reinterpret_cast<uint4*>(dg + p.N) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      }
    }
  } else if constexpr (MODE == kDh) {
    if (!p.sa) {
      float* c = static_cast<float*>(p.c) + (int64_t)m * p.N;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = (j ? nb1 : nb0) + 8 * q + 4 * hi;
          const f32x16_t& r = j ? c1 : c0;
          if (mok && n < p.N)
            *reinterpret_cast<float4*>(c + n) = make_float4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
        }
      return;
    }
    // A result's a and u leave together, without a branch between (each waited for in its turn: the
    // backward pass of 8192 rows, d = 4096, d_ff = 2048, 716 against 709 us; those of both results at once
    // do not fit the registers).
    const int es = p.sca ? 1 : 2, l31 = m - mu;
    const auto ra = rsrc_of(static_cast<const uint8_t*>(p.sa) + (int64_t)mu * p.N * es);
    const auto ru = rsrc_of(static_cast<const uint8_t*>(p.su) + (int64_t)mu * p.N * es);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int nb = j ? nb1 : nb0;
      uint4 va[2], vu[2];  // by pair of quads: after the exchange this lane holds n .. n + 7
      int ea = 0, eu = 0;
      if (p.sca) {
        const auto rsa = rsrc_of(p.sca + (int64_t)mu * (p.N >> 5)), rsu = rsrc_of(p.scu + (int64_t)mu * (p.N >> 5));
        const uint32_t off = mok && nb < p.N ? (uint32_t)(l31 * (p.N >> 5) + (nb >> 5)) : kOOB;
        ea = (int)buf_ld8(rsa, off);
        eu = (int)buf_ld8(rsu, off);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int n = nb + 16 * q + 8 * hi;
          const uint32_t at = mok && n < p.N ? (uint32_t)(l31 * p.N + n) : kOOB;
          const uint2 a = buf_ld8b(ra, at), u = buf_ld8b(ru, at);
          va[q] = make_uint4(a.x, a.y, 0, 0);
          vu[q] = make_uint4(u.x, u.y, 0, 0);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int n = nb + 16 * q + 8 * hi;
          const uint32_t at = mok && n < p.N ? (uint32_t)((l31 * p.N + n) * 2) : kOOB;
          va[q] = buf_ld16(ra, at);
          vu[q] = buf_ld16(ru, at);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const int n = nb + 8 * q + 8 * hi;
        const int64_t at = (int64_t)m * p.N + n;
        float g[8], a[8], u[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t x = __float_as_uint((j ? c1 : c0)[4 * q + e]), y = __float_as_uint((j ? c1 : c0)[4 * q + 4 + e]);
          swap_halves(x, y);
          g[e] = __uint_as_float(x);
          g[4 + e] = __uint_as_float(y);
        }
        const uint4 wa4 = va[q >> 1], wu4 = vu[q >> 1];
        if (p.sca) {
          mx8_values4(wa4.x, ea, a);
          mx8_values4(wa4.y, ea, a + 4);
          mx8_values4(wu4.x, eu, u);
          mx8_values4(wu4.y, eu, u + 4);
        } else {
          const uint32_t wa[4] = {wa4.x, wa4.y, wa4.z, wa4.w}, wu[4] = {wu4.x, wu4.y, wu4.z, wu4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[2 * e] = lo16<H>(wa[e]);
            a[2 * e + 1] = hi16<H>(wa[e]);
            u[2 * e] = lo16<H>(wu[e]);
            u[2 * e + 1] = hi16<H>(wu[e]);
          }
        }
        uint32_t oh[4], oa[4], ou[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const ActD f0 = act_df(a[2 * e], p.act), f1 = act_df(a[2 * e + 1], p.act);
          oh[e] = pack2<H>(f0.f * u[2 * e], f1.f * u[2 * e + 1]);
          oa[e] = pack2<H>(g[2 * e] * u[2 * e] * f0.df, g[2 * e + 1] * u[2 * e + 1] * f1.df);
          ou[e] = pack2<H>(g[2 * e] * f0.f, g[2 * e + 1] * f1.f);
        }
        if (mok && n < p.N) {
          *reinterpret_cast<uint4*>(p.h + at) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
          uint16_t* dg = p.dag + 2 * (int64_t)m * p.N + n;
          *reinterpret_cast<uint4*>(dg) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
          *reinterpret_cast<uint4*>(dg + p.N) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int nb = j ? nb1 : nb0;
      if (MODE == kOut && p.c_f32) {
        float* c = static_cast<float*>(p.c) + (int64_t)m * p.ldc;
        const float* r = static_cast<const float*>(p.res) + (int64_t)m * p.ldr;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = nb + 8 * q + 4 * hi;
          if (mok && n < p.N) {
            float4 v = make_float4((j ? c1 : c0)[4 * q], (j ? c1 : c0)[4 * q + 1], (j ? c1 : c0)[4 * q + 2], (j ? c1 : c0)[4 * q + 3]);
            if (p.res) {
              const float4 o = *reinterpret_cast<const float4*>(r + n);
              v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            *reinterpret_cast<float4*>(c + n) = v;
          }
        }
      } else {
        uint16_t* c = static_cast<uint16_t*>(p.c) + (int64_t)m * p.ldc;
        if (MODE == kDw && m >= p.split) c = static_cast<uint16_t*>(p.c2) + (int64_t)(m - p.split) * p.ldc;
        const uint16_t* r = static_cast<const uint16_t*>(p.res) + (int64_t)m * p.ldr;
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const int n = nb + 8 * q + 8 * hi;
          const bool ok = mok && n < p.N;
          if (MODE == kOut && p.res) {
            // the sum in fp32, then one rounding
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t x = __float_as_uint((j ? c1 : c0)[4 * q + e]), y = __float_as_uint((j ? c1 : c0)[4 * q + 4 + e]);
              swap_halves(x, y);
              v[e] = __uint_as_float(x);
              v[4 + e] = __uint_as_float(y);
            }
            if (ok) {
              const uint4 o = *reinterpret_cast<const uint4*>(r + n);
              const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<H>(v[2 * e] + lo16<H>(ow[e]), v[2 * e + 1] + hi16<H>(ow[e]));
              *reinterpret_cast<uint4*>(c + n) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack2<H>((j ? c1 : c0)[4 * q + 2 * e], (j ? c1 : c0)[4 * q + 2 * e + 1]);
            swap_halves(w[0], w[2]);
            swap_halves(w[1], w[3]);
            if (ok) *reinterpret_cast<uint4*>(c + n) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }
}

// Two 32x32 results of a wave among a piece's sums: 2048 floats, quads of 4 n by lane.
__device__ __forceinline__ void store_part(float* at, const f32x16_t (&c)[2], int lane) {
  float4* d = reinterpret_cast<float4*>(at) + lane;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      d[(j * 4 + q) * 64] = make_float4(c[j][4 * q], c[j][4 * q + 1], c[j][4 * q + 2], c[j][4 * q + 3]);
}
__device__ __forceinline__ void add_part(f32x16_t (&c)[2], const float* at, int lane) {
  const float4* d = reinterpret_cast<const float4*>(at) + lane;
  float4 v[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) v[j][q] = d[(j * 4 + q) * 64];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      c[j][4 * q] += v[j][q].x;
      c[j][4 * q + 1] += v[j][q].y;
      c[j][4 * q + 2] += v[j][q].z;
      c[j][4 * q + 3] += v[j][q].w;
    }
}

template <int MODE, bool H, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, WM* WN / 4) void gemm_kernel(GemmArgs p) {
  constexpr bool AT = MODE == kDw;
  constexpr bool BT = MODE == kDh || MODE == kDx || MODE == kDw;
  constexpr int NW = WM * WN, TM = BM / WM, MT = TM / 32;
  static_assert(BN / WN == 64 && TM % 32 == 0, "a wave computes TM x 64");
  constexpr int ABYTES = BM * 128, BBYTES = BN * 128, SBYTES = ABYTES + BBYTES;
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KB loads a wave issues per stage and operand
  __shared__ __attribute__((aligned(1024))) uint8_t sm[2 * SBYTES];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  const int per_seg = (p.K + 63) >> 6;
  const int stages = MODE == kDx ? 2 * per_seg : per_seg;
  // consecutive blocks share an XCD; `blocks` of them share each tile's stages (rest > 0)
  const int lb = xcd_logical_block(blockIdx.x, gridDim.x);
  const int tile = p.rest ? lb / p.blocks : lb;
  const int s_begin = p.rest ? (lb - tile * p.blocks) * p.per : 0;
  const int s_end = p.rest ? min(stages, s_begin + p.per) : stages;
  const TilePos tp = tile_pos(p, tile);
  const int m0 = tp.m * BM, n0 = tp.n * (kBeside<MODE> ? BN / 2 : BN);

  // ---- loads: per-lane byte offsets within the tile, from a base that moves with k ----
  uint32_t offA[LA], offB[LB];
  int kA[LA], kB[LB];  // first k of the piece within the stage
#pragma unroll
  for (int j = 0; j < LA; ++j) {
    const int q = (wave * LA + j) * 64 + lane;
    if constexpr (!AT) {
      const int r = q >> 3, pc = (q & 7) ^ ((r >> 1) & 7);
      kA[j] = pc * 8;
      offA[j] = m0 + r < p.M ? (uint32_t)(r * p.lda * 2 + pc * 16) : kOOB;
    } else {
      constexpr int PR = BM / 8;
      const int k = q / PR, pc = (q % PR) ^ ((k & 3) << 2);
      kA[j] = k;
      offA[j] = m0 + pc * 8 < p.M ? (uint32_t)(k * p.lda * 2 + pc * 16) : kOOB;
    }
  }
#pragma unroll
  for (int j = 0; j < LB; ++j) {
    const int q = (wave * LB + j) * 64 + lane;
    if constexpr (!BT) {
      const int r = q >> 3, pc = (q & 7) ^ ((r >> 1) & 7);
      const int n = kBeside<MODE> ? (r >> 6) * 32 + (r & 31) : r;
      kB[j] = pc * 8;
      offB[j] = n0 + n < p.N ? (uint32_t)(n * p.ldb * 2 + pc * 16) : kOOB;
    } else {
      constexpr int PR = BN / 8;
      const int k = q / PR, pc = (q % PR) ^ ((k & 3) << 2);
      kB[j] = k;
      offB[j] = n0 + pc * 8 < p.N ? (uint32_t)(k * p.ldb * 2 + pc * 16) : kOOB;
    }
  }

  const uint32_t sm0 = lds_addr(sm);

  auto load_stage = [&](int s) {
    int k0 = s << 6;
    const uint16_t *pa = p.a, *pb = p.b;
    if (MODE == kDx && s >= per_seg) {
      k0 = (s - per_seg) << 6;
      pa = p.a + p.K;
      pb = p.b2;
    }
    const int left = p.K - k0;
    const uint32_t dst = sm0 + (s & 1) * SBYTES;
    const auto ra = rsrc_of(AT ? pa + k0 * p.lda + m0 : pa + m0 * p.lda + k0);
#pragma unroll
    for (int j = 0; j < LA; ++j)
      lds_load16(ra, kA[j] < left ? offA[j] : kOOB, 0, dst + (wave * LA + j) * 1024);
    if constexpr (kBeside<MODE>) {
#pragma unroll
      for (int j = 0; j < LB; ++j) {
        // 8 rows of one matrix: blocks of 32 rows alternate between Wg and Wu
        const uint16_t* w = ((wave * LB + j) & 4) ? p.b2 : p.b;
        lds_load16(rsrc_of(w + n0 * p.ldb + k0), kB[j] < left ? offB[j] : kOOB, 0, dst + ABYTES + (wave * LB + j) * 1024);
      }
    } else {
      const auto rb = rsrc_of(BT ? pb + k0 * p.ldb + n0 : pb + n0 * p.ldb + k0);
#pragma unroll
      for (int j = 0; j < LB; ++j)
        lds_load16(rb, kB[j] < left ? offB[j] : kOOB, 0, dst + ABYTES + (wave * LB + j) * 1024);
    }
  };

  // ---- fragments ----
  const int hi = lane >> 5, l31 = lane & 31;
  // along k: row l31 of the subtile, piece (2 slice + hi) ^ (row / 2 & 7)
  auto frag_k = [&](const uint8_t* base, int row, int slice) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(base + (row + l31) * 128 + (((2 * slice + hi) ^ ((l31 >> 1) & 7)) << 4));
  };
  // transposed: rows k = 16 slice + 8 hi + {0, 4} + kk, columns 16 ((lane >> 4) & 1) + 4 (lane & 3)
  const int kk = (lane >> 2) & 3;
  auto frag_t = [&](const uint8_t* base, int width, int col, int slice) -> i32x4_t {
    const int pc = ((col >> 3) ^ (kk << 2)) + ((lane >> 3) & 2) + ((lane >> 1) & 1);
    const uint8_t* q = base + (16 * slice + 8 * hi + kk) * width * 2 + pc * 16 + (lane & 1) * 8;
    typedef const __attribute__((address_space(3))) s16x4_t* lp;
    const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(lp)q);
    const s16x4_t v1 =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(lp)(q + 4 * width * 2));
    const u32x2_t a = __builtin_bit_cast(u32x2_t, v0), b = __builtin_bit_cast(u32x2_t, v1);
    return i32x4_t{(int)a.x, (int)a.y, (int)b.x, (int)b.y};
  };

  f32x16_t acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x16_t{};

  if (s_begin < s_end) load_stage(s_begin);
  for (int s = s_begin; s < s_end; ++s) {
    // this wave's loads of stage s have landed; past the barrier everyone's have, and nobody
    // reads the other buffer any more
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 1 < s_end) load_stage(s + 1);
    const uint8_t* sa = sm + (s & 1) * SBYTES;
    const uint8_t* sb = sa + ABYTES;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      i32x4_t fa[MT], fb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        fb[j] = BT ? frag_t(sb, BN, wn * 64 + j * 32, k) : frag_k(sb, wn * 64 + j * 32, k);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i] = AT ? frag_t(sa, BM, wm * TM + i * 32, k) : frag_k(sa, wm * TM + i * 32, k);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32<H>(fb[j], fa[i], acc[i][j]);
    }
    // the reads above are done before anyone passes the next barrier
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (p.rest) {
      store_part(p.part + (size_t)lb * (BM * BN) + (wave * MT + i) * 2 * 1024, acc[i], lane);
    } else {
      const int nb = n0 + wn * (kBeside<MODE> ? 32 : 64);
      const int m = m0 + wm * TM + i * 32;
      epilogue<MODE, H>(p, acc[i][0], acc[i][1], m, m + l31, nb, nb + 32, hi);
    }
  }
}

// The shared tiles of the kernel above: sums in the order of k, then the epilogue.  A block per tile and
// 32-row piece of the waves.
template <int MODE, bool H, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void gemm_join_kernel(GemmArgs p) {
  constexpr int TM = BM / WM, MT = TM / 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, t = blockIdx.x / MT, i = blockIdx.x % MT;
  const TilePos tp = tile_pos(p, t);
  const int m = tp.m * BM + wm * TM + i * 32;
  if (m >= p.M) return;
  f32x16_t acc[2] = {f32x16_t{}, f32x16_t{}};
  for (int b = 0; b < p.blocks; ++b)
    add_part(acc, p.part + (size_t)(t * p.blocks + b) * (BM * BN) + (wave * MT + i) * 2 * 1024, lane);
  const int nb = tp.n * (kBeside<MODE> ? BN / 2 : BN) + wn * (kBeside<MODE> ? 32 : 64);
  epilogue<MODE, H>(p, acc[0], acc[1], m, m + (lane & 31), nb, nb + 32, lane >> 5);
}

// The same product on 256 x 256 tiles, for results large enough to fill the chip with them.
// 8 waves, two per SIMD; each computes 64 rows and 32 columns of every 128 x 128 quarter.  A
// stage of 64 k is four regions of 16 KB (the two halves of A's rows and of B's), two stages
// in LDS.  A stage is two steps, one per half of A's rows: a read section (fragments from LDS, loads
// into regions that everyone has read) and a multiply section (16 MFMAs), each closed by a
// barrier.  The waves 4..7 run one section behind the waves 0..3, so on every SIMD one
// wave multiplies while the other reads.  Sections t = 0..3 of stage s for the first group (the
// second does the same one later):
//   t = 0  read A0, B0, B1 of s; load A1 of s + 1; wait for A1 of s
//   t = 1  A0 x B0, A0 x B1
//   t = 2  read A1 of s; load A0, B0, B1 of s + 2; wait for A0, B0, B1 of s + 1
//   t = 3  A1 x B1, A1 x B0
// A region is loaded again two sections after the first group read it, one after the second did
// (both end a read section with their reads done): A1 of s + 1 goes where A1 of s - 1 was read at t = -2
// and -1.  It is waited for by both groups at least one barrier before its first read, and has six
// sections to arrive.  Loads past the last stage are masked (they write zeros nobody reads), which keeps
// the counts of the waits.  (Four steps of a quarter each, with 8 MFMAs a section, took 4 % longer.)
// MH: halves of A's rows, 2 as above or 1 (tiles of 128 x 256 for fewer rows: a stage is one step of A0, B0
// and B1, three stages lie in LDS, and the loads of stage s + 2 go where stage s - 1 was read).
template <int MODE, bool H, int MH>
__global__ __launch_bounds__(512, 2) void gemm256_kernel(GemmArgs p) {
  constexpr bool AT = MODE == kDw;
  constexpr bool BT = MODE == kDh || MODE == kDx || MODE == kDw;
  constexpr int REG = 16384;
  enum { A0 = 0, B0 = REG, B1 = 2 * REG, A1 = 3 * REG, STAGE = (2 + MH) * REG, PLACES = MH == 2 ? 2 : 3 };
  __shared__ __attribute__((aligned(1024))) uint8_t sm[PLACES * STAGE];
  constexpr int BM = 128 * MH, PART = BM * 256;  // rows of a tile, floats of its sums

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;

  const int hi = lane >> 5, l31 = lane & 31, kk = (lane >> 2) & 3;
  const int per_seg = (p.K + 63) >> 6;
  const int stages = MODE == kDx ? 2 * per_seg : per_seg;

  // This block's piece of work: a whole tile, or stages [at, end) of the rest's, which touch at
  // most two tiles (per < stages).
  int tile, at = 0, end = 1, b = 0;
  const bool piece = (int)blockIdx.x >= p.whole;
  if (!piece) {
    tile = xcd_logical_block(blockIdx.x, p.whole);
  } else {
    b = xcd_logical_block(blockIdx.x - p.whole, p.parts);
    const int g = b / p.blocks, line = p.group * stages;
    at = g * line + (b - g * p.blocks) * p.per;
    end = min(min(at + p.per, (g + 1) * line), p.rest * stages);
    tile = p.whole;
  }
  while (at < end) {
    int s_begin = 0, s_end = stages, slot = -1;
    if (piece) {
      const int t = at / stages;
      tile = p.whole + t;
      s_begin = at - t * stages;
      s_end = min(stages, end - t * stages);
      if (s_end - s_begin < stages) slot = b + t;
      at = t * stages + s_end;
    } else {
      at = end;
    }
    const TilePos tp = tile_pos(p, tile);
    const int m0 = tp.m * BM, n0 = tp.n * (kBeside<MODE> ? 128 : 256);
    // rows of a wave in the two halves: those past the end are neither read nor multiplied
    const bool any[2] = {m0 + wm * 64 < p.M, m0 + 128 + wm * 64 < p.M};

    // ---- loads: a wave brings chunks 2 wave and 2 wave + 1 (1 KB) of every region ----
    uint32_t offA[MH][2], offB[2][2];  // [half][chunk]
    int kA[2], kB[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = wave * 2 + j;
      const int r = c * 8 + (lane >> 3), pk = (lane & 7) ^ ((r >> 1) & 7);        // along k
      const int kt = c * 4 + (lane >> 4), pt = (lane & 15) ^ ((lane >> 4) << 2);  // transposed
      kA[j] = AT ? kt : pk * 8;
      kB[j] = BT ? kt : pk * 8;
#pragma unroll
      for (int h = 0; h < MH; ++h) {
        if constexpr (AT)
          offA[h][j] = m0 + h * 128 + pt * 8 < p.M ? (uint32_t)(kt * p.lda * 2 + pt * 16) : kOOB;
        else
          offA[h][j] = m0 + h * 128 + r < p.M ? (uint32_t)(r * p.lda * 2 + pk * 16) : kOOB;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int nh = n0 + (kBeside<MODE> ? 0 : h * 128);
        if constexpr (BT)
          offB[h][j] = nh + pt * 8 < p.N ? (uint32_t)(kt * p.ldb * 2 + pt * 16) : kOOB;
        else
          offB[h][j] = nh + r < p.N ? (uint32_t)(r * p.ldb * 2 + pk * 16) : kOOB;
      }
    }
    // Each region's source moves on by a stage per load.
    const uint32_t sm0 = lds_addr(sm) + wave * 2048;
    const int64_t step_a = AT ? p.lda * 128 : 128, step_b = BT ? p.ldb * 128 : 128;  // bytes
    auto first_a = [&](int h) -> const uint8_t* {
      const bool two = MODE == kDx && s_begin >= per_seg;
      const int k0 = (s_begin - (two ? per_seg : 0)) << 6, m = m0 + h * 128;
      const uint16_t* a = p.a + (two ? p.K : 0);
      return reinterpret_cast<const uint8_t*>(AT ? a + k0 * p.lda + m : a + m * p.lda + k0);
    };
    auto first_b = [&](int h) -> const uint8_t* {
      const bool two = MODE == kDx && s_begin >= per_seg;
      const int k0 = (s_begin - (two ? per_seg : 0)) << 6, n = n0 + (kBeside<MODE> ? 0 : h * 128);
      const uint16_t* b = two || (kBeside<MODE> && h) ? p.b2 : p.b;
      return reinterpret_cast<const uint8_t*>(BT ? b + k0 * p.ldb + n : b + n * p.ldb + k0);
    };
    const uint8_t *pa[2] = {first_a(0), first_a(1)}, *pb[2] = {first_b(0), first_b(1)};
    auto k_left = [&](int s) {
      if (s >= s_end) return 0;
      return p.K - ((MODE == kDx && s >= per_seg ? s - per_seg : s) << 6);
    };
    auto load_a = [&](int s, int h, int place) {
      if (MODE == kDx && s == per_seg && s != s_begin)
        pa[h] = reinterpret_cast<const uint8_t*>(p.a + p.K + (m0 + h * 128) * p.lda);
      const int left = k_left(s);
      const auto rs = rsrc_of(pa[h]);
      const uint32_t dst = sm0 + place * STAGE + (h ? A1 : A0);
#pragma unroll
      for (int j = 0; j < 2; ++j) lds_load16(rs, kA[j] < left ? offA[h][j] : kOOB, 0, dst + j * 1024);
      pa[h] += step_a;
    };
    auto load_b = [&](int s, int h, int place) {
      if (MODE == kDx && s == per_seg && s != s_begin) pb[h] = reinterpret_cast<const uint8_t*>(p.b2 + n0 + h * 128);
      const int left = k_left(s);
      const auto rs = rsrc_of(pb[h]);
      const uint32_t dst = sm0 + place * STAGE + (h ? B1 : B0);
#pragma unroll
      for (int j = 0; j < 2; ++j) lds_load16(rs, kB[j] < left ? offB[h][j] : kOOB, 0, dst + j * 1024);
      pb[h] += step_b;
    };

    // ---- fragments of a region: 32 rows (or columns) from `row`, slice of 16 k ----
    auto frag_k = [&](const uint8_t* base, int row, int slice) -> i32x4_t {
      return *reinterpret_cast<const i32x4_t*>(base + (row + l31) * 128 + (((2 * slice + hi) ^ ((l31 >> 1) & 7)) << 4));
    };
    auto frag_t = [&](const uint8_t* base, int col, int slice) -> i32x4_t {
      const int pc = ((col >> 3) ^ (kk << 2)) + ((lane >> 3) & 2) + ((lane >> 1) & 1);
      const uint8_t* q = base + (16 * slice + 8 * hi + kk) * 256 + pc * 16 + (lane & 1) * 8;
      typedef __attribute__((address_space(3))) s16x4_t* lp;
      const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)q));
      const u32x2_t b = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(q + 1024)));
      return i32x4_t{(int)a.x, (int)a.y, (int)b.x, (int)b.y};
    };

    f32x16_t acc[2 * MH][2];  // [2 half + 32-row piece][half of the columns]
#pragma unroll
    for (int i = 0; i < 2 * MH; ++i) acc[i][0] = acc[i][1] = f32x16_t{};
    i32x4_t fa[2][4], fb0[4], fb1[4];

    auto read_a = [&](const uint8_t* base) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          fa[i][k] = AT ? frag_t(base, wm * 64 + i * 32, k) : frag_k(base, wm * 64 + i * 32, k);
    };
    auto read_b = [&](const uint8_t* base, i32x4_t (&f)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = BT ? frag_t(base, wn * 32, k) : frag_k(base, wn * 32, k);
    };
    auto multiply = [&](int half) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[2 * half + i][0] = mfma32<H>(fb0[k], fa[i][k], acc[2 * half + i][0]);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[2 * half + i][1] = mfma32<H>(fb1[k], fa[i][k], acc[2 * half + i][1]);
      }
      __builtin_amdgcn_s_setprio(0);
    };
    // The end of a section: nothing moves across.
    auto meet = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto reads_done = [&]() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };

    if (s_begin < s_end) {
      load_a(s_begin, 0, 0);
      load_b(s_begin, 0, 0);
      load_b(s_begin, 1, 0);
      if constexpr (MH == 2) load_a(s_begin, 1, 0);
      load_a(s_begin + 1, 0, 1);
      load_b(s_begin + 1, 0, 1);
      load_b(s_begin + 1, 1, 1);
      constexpr int WAIT = MH == 2 ? 8 : 6;
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(WAIT) : "memory");  // A0, B0 and B1 of the first stage
      meet();
      if (wm) meet();
      // RAGGED: the tile has rows past the end.  Asking at every step would cost a whole tile 4 %.
      auto walk = [&](auto ragged) {
        constexpr bool RAGGED = decltype(ragged)::value;
        int here = 0;
        for (int s = s_begin; s < s_end; ++s) {
          const uint8_t* st = sm + here * STAGE;
          const int other = here == 0 ? PLACES - 1 : here - 1;
          if (!RAGGED || any[0]) read_a(st + A0);
          read_b(st + B0, fb0);
          read_b(st + B1, fb1);
          if constexpr (MH == 2) {
            load_a(s + 1, 1, other);
            reads_done();
            asm volatile("s_waitcnt vmcnt(8)" ::: "memory");  // A1 of this stage
          } else {
            load_a(s + 2, 0, other);
            load_b(s + 2, 0, other);
            load_b(s + 2, 1, other);
            reads_done();
            asm volatile("s_waitcnt vmcnt(6)" ::: "memory");  // the next stage
          }
          meet();
          if (!RAGGED || any[0]) multiply(0);
          meet();
          if constexpr (MH == 2) {
            if (!RAGGED || any[1]) read_a(st + A1);
            load_a(s + 2, 0, here);
            load_b(s + 2, 0, here);
            load_b(s + 2, 1, here);
            reads_done();
            asm volatile("s_waitcnt vmcnt(8)" ::: "memory");  // A0, B0 and B1 of the next stage
            meet();
            if (!RAGGED || any[1]) multiply(1);
            meet();
          }
          here = here == PLACES - 1 ? 0 : here + 1;
        }
      };
      if (m0 + BM - 64 < p.M)
        walk(std::false_type{});
      else
        walk(std::true_type{});
      if (!wm) meet();
      // the masked loads' writes too: a wave's next loads go where its own last ones went
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

#pragma unroll
    for (int i = 0; i < 2 * MH; ++i) {
      if (slot >= 0) {
        if (m0 + (i >> 1) * 128 + wm * 64 + (i & 1) * 32 < p.M)
          store_part(p.part + (size_t)slot * PART + (wave * 2 * MH + i) * 2048, acc[i], lane);
      } else {
        const int m = m0 + (i >> 1) * 128 + wm * 64 + (i & 1) * 32;
        const int nb = n0 + wn * 32;
        epilogue<MODE, H>(p, acc[i][0], acc[i][1], m, m + l31, nb, nb + 128, hi);
      }
    }
  }
}

// The tiles whose stages several blocks shared: their sums, always added in the order of k, then the
// epilogue.  A block per tile and 32-row piece of the waves; bound by memory (256 KB a part and tile).
template <int MODE, bool H, int MH>
__global__ __launch_bounds__(512) void gemm256_join_kernel(GemmArgs p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, i = blockIdx.x % (2 * MH), t = blockIdx.x / (2 * MH);
  const int stages = (MODE == kDx ? 2 : 1) * ((p.K + 63) >> 6);
  const int g = t / p.group, from = (t - g * p.group) * stages;
  const int first = g * p.blocks + from / p.per, last = g * p.blocks + (from + stages - 1) / p.per;
  if (first == last) return;  // one block had it all
  const TilePos tp = tile_pos(p, p.whole + t);
  const int m = tp.m * 128 * MH + (i >> 1) * 128 + wm * 64 + (i & 1) * 32;
  if (m >= p.M) return;
  f32x16_t acc[2] = {f32x16_t{}, f32x16_t{}};
  for (int b = first; b <= last; ++b) add_part(acc, p.part + (size_t)(b + t) * (MH * 128 * 256) + (wave * 2 * MH + i) * 2048, lane);
  const int nb = tp.n * (kBeside<MODE> ? 128 : 256) + wn * 32;
  epilogue<MODE, H>(p, acc[0], acc[1], m, m + (lane & 31), nb, nb + 128, lane >> 5);
}

// ---- few rows: the weights stream once ------------------------------------------------
// y[t, n] = sum over k of x[t, k] W[n, k] for up to 16 * NT rows.  A block owns 16 weight rows
// (GU: 8 rows of Wg and the same 8 of Wu), its waves split k in steps of 64 and add their
// parts in LDS in a fixed order.  v_mfma_f32_16x16x32: the weights are the second operand, so
// each element is loaded once, straight into registers; rows of x past T repeat the last one
// and their sums are dropped.
struct SkinnyArgs {
  const uint16_t *x, *w, *w2;
  int64_t ldx;
  int T, K, N;
  int act;
  uint16_t* h;  // GU
  void* c;      // else
  int64_t ldc;
  int c_f32;
  const void* res;
  int64_t ldr;
};

template <bool GU, bool H, int NT, int W>
__global__ __launch_bounds__(64 * W) void skinny_kernel(SkinnyArgs p) {
  constexpr int RB = GU ? 8 : 16, U = NT <= 2 ? 4 : 2;
  __shared__ float red[W][NT * 16][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * RB, t0 = blockIdx.y * (16 * NT);
  const int row = r0 + (GU ? (n & 7) : n);
  const uint16_t* wp = GU && n >= 8 ? p.w2 : p.w;
  wp += (int64_t)min(row, p.N - 1) * p.K;
  const uint16_t* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xp[i] = p.x + (int64_t)min(t0 + i * 16 + n, p.T - 1) * p.ldx;
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{};
  const int steps = (p.K + 31) >> 5;  // of 32 k; pairs of steps go to the waves in turn
  for (int s0 = 2 * wave; s0 < steps; s0 += 2 * W * (U / 2)) {
    i32x4_t fw[U], fx[U][NT];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int s = s0 + (v >> 1) * 2 * W + (v & 1);
      const int k = s * 32 + g * 8;
      const bool ok = k < p.K;  // K % 8 == 0
      const int ka = ok ? k : 0;
      fw[v] = *reinterpret_cast<const i32x4_t*>(wp + ka);
#pragma unroll
      for (int i = 0; i < NT; ++i) fx[v][i] = *reinterpret_cast<const i32x4_t*>(xp[i] + ka);
      if (!ok) {
        fw[v] = i32x4_t{};
#pragma unroll
        for (int i = 0; i < NT; ++i) fx[v][i] = i32x4_t{};
      }
    }
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = mfma16<H>(fx[v][i], fw[v], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][i * 16 + g * 4 + r][n] = acc[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 16 * RB; e += 64 * W) {
    const int t = e / RB, c = e % RB;
    const int tt = t0 + t, nn = r0 + c;
    if (tt >= p.T || nn >= p.N) continue;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][t][c];
    if constexpr (GU) {
      float u = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) u += red[w][t][c + 8];
      const float v = act_f(s, p.act) * u;
      p.h[(int64_t)tt * p.N + nn] = (uint16_t)pack2<H>(v, 0.0f);
    } else if (p.c_f32) {
      if (p.res) s += static_cast<const float*>(p.res)[(int64_t)tt * p.ldr + nn];
      static_cast<float*>(p.c)[(int64_t)tt * p.ldc + nn] = s;
    } else {
      if (p.res) s += to_f32<H>(static_cast<const uint16_t*>(p.res)[(int64_t)tt * p.ldr + nn]);
      static_cast<uint16_t*>(p.c)[(int64_t)tt * p.ldc + nn] = (uint16_t)pack2<H>(s, 0.0f);
    }
  }
}

// ---- 8-bit activations --------------------------------------------------------------
// One thread per 16 elements (half a block of 32): 32 bytes in, 16 out, the block's largest by one
// exchange with its neighbour; bound by memory (8192 x 4096: 17-18 us, 5.6-6.0 TB/s; unpacking 19-20 us, 5.1-5.4 TB/s).
__device__ __forceinline__ int64_t act8_row() {
  return ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.y + threadIdx.y;
}
template <bool H>
__global__ __launch_bounds__(256) void act8_pack_kernel(const uint16_t* src, int64_t ld, int rows, int n,
                                                        uint8_t* codes, uint8_t* scales) {
  const int64_t row = act8_row();
  if (row >= rows) return;  // a row's two halves of a block always stay together
  for (int c = threadIdx.x; c < n / 16; c += blockDim.x) {
    const uint4* q = reinterpret_cast<const uint4*>(src + row * ld + c * 16);
    const uint4 v0 = q[0], v1 = q[1];
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    float f[16];
    float am = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[2 * e] = lo16<H>(w[e]);
      f[2 * e + 1] = hi16<H>(w[e]);
      am = fmaxf(am, fmaxf(fin_abs(f[2 * e]), fin_abs(f[2 * e + 1])));
    }
    am = fmaxf(am, __shfl_xor(am, 1, WAVE));
    const int sc = mx8_scale(am);
    *reinterpret_cast<uint4*>(codes + row * n + c * 16) =
        make_uint4(mx8_codes4(f[0], f[1], f[2], f[3], sc), mx8_codes4(f[4], f[5], f[6], f[7], sc),
                   mx8_codes4(f[8], f[9], f[10], f[11], sc), mx8_codes4(f[12], f[13], f[14], f[15], sc));
    if ((c & 1) == 0) scales[row * (n / 32) + c / 2] = (uint8_t)sc;
  }
}
// FIT: values past the type's end become its largest (fp16 always, bf16 for a backward pass); else infinities.
template <bool H, bool FIT>
__global__ __launch_bounds__(256) void act8_unpack_kernel(const uint8_t* codes, const uint8_t* scales, int rows, int n,
                                                          uint16_t* dst, int64_t ld) {
  const int64_t row = act8_row();
  if (row >= rows) return;
  for (int c = threadIdx.x; c < n / 16; c += blockDim.x) {
    const uint4 v = *reinterpret_cast<const uint4*>(codes + row * n + c * 16);
    const int sc = scales[row * (n / 32) + c / 2];
    float f[16];
    mx8_values4(v.x, sc, f);
    mx8_values4(v.y, sc, f + 4);
    mx8_values4(v.z, sc, f + 8);
    mx8_values4(v.w, sc, f + 12);
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e] = FIT ? pack2<H>(fit16<H>(f[2 * e]), fit16<H>(f[2 * e + 1])) : pack2<H>(f[2 * e], f[2 * e + 1]);
    uint4* q = reinterpret_cast<uint4*>(dst + row * ld + c * 16);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ---- launches -------------------------------------------------------------------------

template <int MODE, bool H>
int gemm_go(GemmArgs& A, hipStream_t s) {
  const int64_t n = kBeside<MODE> ? 2 * (int64_t)A.N : A.N;
  const Cut c = cut_of(A.M, n, (MODE == kDx ? 2 : 1) * ((A.K + 63) / 64));
  A.tiles_m = c.tiles_m;
  A.tiles_n = c.tiles_n;
  A.whole = c.whole;
  A.rest = c.rest;
  A.group = c.group;
  A.blocks = c.blocks;
  A.per = c.per;
  A.parts = c.parts;
  if (A.tiles_m == 0 || A.tiles_n == 0) return FT_OK;
  if ((int64_t)A.tiles_m * A.tiles_n > 0x7ffffff) return fail(FT_EINVAL, "gated_ffn: too many tiles");
  if (c.tile == 256) {
    hipLaunchKernelGGL((gemm256_kernel<MODE, H, 2>), dim3((unsigned)(c.whole + c.parts)), dim3(512), 0, s, A);
    if (c.rest) hipLaunchKernelGGL((gemm256_join_kernel<MODE, H, 2>), dim3((unsigned)c.rest * 4), dim3(512), 0, s, A);
  } else if (c.tile == 384) {
    hipLaunchKernelGGL((gemm256_kernel<MODE, H, 1>), dim3((unsigned)(c.whole + c.parts)), dim3(512), 0, s, A);
    if (c.rest) hipLaunchKernelGGL((gemm256_join_kernel<MODE, H, 1>), dim3((unsigned)c.rest * 2), dim3(512), 0, s, A);
  } else {
    hipLaunchKernelGGL((gemm_kernel<MODE, H, 128, 128, 2, 2>), dim3((unsigned)c.parts), dim3(256), 0, s, A);
    if (c.rest)
      hipLaunchKernelGGL((gemm_join_kernel<MODE, H, 128, 128, 2, 2>), dim3((unsigned)c.rest * 2), dim3(256), 0, s, A);
  }
  return launched("gemm_kernel");
}

template <int MODE>
int gemm_launch(GemmArgs& A, bool half, hipStream_t s) {
  return half ? gemm_go<MODE, true>(A, s) : gemm_go<MODE, false>(A, s);
}

template <bool GU, bool H>
int skinny_go(SkinnyArgs& A, hipStream_t s) {
  constexpr int RB = GU ? 8 : 16;
  const unsigned nb = (unsigned)((A.N + RB - 1) / RB);
  // (one token, d = 4096, d_ff = 2048, both products: 13.1 us with 16 waves, 14.5 us with 8)
  if (A.T <= 16)
    hipLaunchKernelGGL((skinny_kernel<GU, H, 1, 16>), dim3(nb, 1), dim3(1024), 0, s, A);
  else if (A.T <= 32)
    hipLaunchKernelGGL((skinny_kernel<GU, H, 2, 8>), dim3(nb, 1), dim3(512), 0, s, A);
  else
    hipLaunchKernelGGL((skinny_kernel<GU, H, 4, 8>), dim3(nb, (unsigned)((A.T + 63) / 64)), dim3(512), 0, s, A);
  return launched("skinny_kernel");
}

}  // namespace

int launch_gated_ffn(const DenseFfn& F, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool half = F.dtype == FT_T_FP16;
  if (F.T <= 0) return FT_OK;
  if (gated_ffn_streams(F.T, F.save_fmt)) {
    SkinnyArgs A{};
    A.x = F.x;
    A.ldx = F.ldx;
    A.w = F.wg;
    A.w2 = F.wu;
    A.T = F.T;
    A.K = F.d;
    A.N = F.d_ff;
    A.act = F.act;
    A.h = F.h;
    int st = half ? skinny_go<true, true>(A, s) : skinny_go<true, false>(A, s);
    if (st) return st;
    SkinnyArgs D{};
    D.x = F.h;
    D.ldx = F.d_ff;
    D.w = F.wd;
    D.T = F.T;
    D.K = F.d_ff;
    D.N = F.d;
    D.c = F.y;
    D.ldc = F.ldy;
    D.c_f32 = F.y_f32;
    D.res = F.res;
    D.ldr = F.ldr;
    return half ? skinny_go<false, true>(D, s) : skinny_go<false, false>(D, s);
  }
  GemmArgs A{};
  A.part = F.part;
  A.a = F.x;
  A.lda = F.ldx;
  A.b = F.wg;
  A.b2 = F.wu;
  A.ldb = F.d;
  A.M = F.T;
  A.N = F.d_ff;
  A.K = F.d;
  A.act = F.act;
  A.h = F.h;
  A.sa = F.sa;
  A.su = F.su;
  A.sca = F.sca;
  A.scu = F.scu;
  int st = gemm_launch<kGateUp>(A, half, s);
  if (st) return st;
  GemmArgs D{};
  D.part = F.part;
  D.a = F.h;
  D.lda = F.d_ff;
  D.b = F.wd;
  D.ldb = F.d_ff;
  D.M = F.T;
  D.N = F.d;
  D.K = F.d_ff;
  D.c = F.y;
  D.ldc = F.ldy;
  D.c_f32 = F.y_f32;
  D.res = F.res;
  D.ldr = F.ldr;
  return gemm_launch<kOut>(D, half, s);
}

int launch_gated_ffn_bwd(const DenseFfn& F, const DenseGrad& G, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool half = F.dtype == FT_T_FP16;
  int st;
  if (F.T > 0) {
    GemmArgs A{};
    A.part = F.part;
    A.a = G.dy;
    A.lda = G.lddy;
    A.b = F.wd;
    A.ldb = F.d_ff;
    A.M = F.T;
    A.N = F.d_ff;
    A.K = F.d;
    A.act = F.act;
    A.sa = F.sa;
    A.su = F.su;
    A.sca = F.sca;
    A.scu = F.scu;
    A.h = F.h;
    A.dag = G.dag;
    A.c = G.dh;
    if ((st = gemm_launch<kDh>(A, half, s))) return st;
    if (!F.sa) {
      // a and u again, in fp32 where they are used: rounded to 16 bits on the way they would double
      // the gradients' error
      GemmArgs B{};
      B.part = F.part;
      B.a = F.x;
      B.lda = F.ldx;
      B.b = F.wg;
      B.b2 = F.wu;
      B.ldb = F.d;
      B.M = F.T;
      B.N = F.d_ff;
      B.K = F.d;
      B.act = F.act;
      B.c = G.dh;
      B.h = F.h;
      B.dag = G.dag;
      if ((st = gemm_launch<kAgain>(B, half, s))) return st;
    }
  }
  if (G.dwd) {
    GemmArgs A{};
    A.part = F.part;
    A.a = G.dy;
    A.lda = G.lddy;
    A.b = F.h;
    A.ldb = F.d_ff;
    A.M = F.d;
    A.N = F.d_ff;
    A.K = F.T;
    A.c = G.dwd;
    A.ldc = F.d_ff;
    A.split = F.d;
    if ((st = gemm_launch<kDw>(A, half, s))) return st;
    GemmArgs B{};
    B.part = F.part;
    B.a = G.dag;
    B.lda = 2 * (int64_t)F.d_ff;
    B.b = F.x;
    B.ldb = F.ldx;
    B.M = 2 * F.d_ff;
    B.N = F.d;
    B.K = F.T;
    B.c = G.dwg;
    B.c2 = G.dwu;
    B.ldc = F.d;
    B.split = F.d_ff;
    if ((st = gemm_launch<kDw>(B, half, s))) return st;
  }
  if (G.dx && F.T > 0) {
    GemmArgs A{};
    A.part = F.part;
    A.a = G.dag;
    A.lda = 2 * (int64_t)F.d_ff;
    A.b = F.wg;
    A.b2 = F.wu;
    A.ldb = F.d;
    A.M = F.T;
    A.N = F.d;
    A.K = F.d_ff;
    A.c = G.dx;
    A.ldc = G.lddx;
    if ((st = gemm_launch<kDx>(A, half, s))) return st;
  }
  return FT_OK;
}

static dim3 act8_block(int n) {
  unsigned x = 2;
  while (x < 256 && (int)x < n / 16) x *= 2;
  return dim3(x, 256 / x);
}
// Blocks for `rows` in two dimensions: a grid's first one holds fewer than 2^32 threads.
static dim3 act8_grid(int rows, unsigned per) {
  const unsigned n = ((unsigned)rows + per - 1) / per, x = n < 65536 ? n : 65536;
  return dim3(x, (n + x - 1) / x);
}

int launch_act8_pack(const uint16_t* src, int64_t ld, int rows, int n, bool half, uint8_t* codes, uint8_t* scales,
                     void* stream) {
  if (rows <= 0) return FT_OK;
  const dim3 b = act8_block(n), g = act8_grid(rows, b.y);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (half)
    hipLaunchKernelGGL(act8_pack_kernel<true>, g, b, 0, s, src, ld, rows, n, codes, scales);
  else
    hipLaunchKernelGGL(act8_pack_kernel<false>, g, b, 0, s, src, ld, rows, n, codes, scales);
  return launched("act8_pack_kernel");
}
int launch_act8_unpack(const uint8_t* codes, const uint8_t* scales, int rows, int n, bool half, bool fit,
                       uint16_t* dst, int64_t ld, void* stream) {
  if (rows <= 0) return FT_OK;
  const dim3 b = act8_block(n), g = act8_grid(rows, b.y);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (half)
    hipLaunchKernelGGL((act8_unpack_kernel<true, true>), g, b, 0, s, codes, scales, rows, n, dst, ld);
  else if (fit)
    hipLaunchKernelGGL((act8_unpack_kernel<false, true>), g, b, 0, s, codes, scales, rows, n, dst, ld);
  else
    hipLaunchKernelGGL((act8_unpack_kernel<false, false>), g, b, 0, s, codes, scales, rows, n, dst, ld);
  return launched("act8_unpack_kernel");
}

}  // namespace ft

// Products with 4-bit weights and group scales, for few tokens.  gfx950 only.
//
//   y[t, n] = sum over groups g of scale[n, g] * sum over k in g of (code[n, k] - zero[n, g]) x[t, k]
//
// A block owns 16 weight rows (a gate/up product: 8 rows of each matrix); its waves take
// chunks of 128 k in turn and add their parts in LDS in a fixed order.  A lane loads 32
// codes of one row (16 bytes); two exchanges across the wave's four row groups (permlane32
// and permlane16 swaps) turn these into the operands of four v_mfma_f32_16x16x32, each of 32
// consecutive k, so a group of 32, 64 or 128 is one, two or four whole MFMAs.
//
// A code becomes the exact 16-bit float 16 + code by placing its 4 bits into the mantissa of
// 16.0: a shift and an and-or for two codes.  A second MFMA on the constant -(16 + zero), which
// is exact too, takes the offset away again within the same fp32 sum; the matrix cores are
// idle in this memory-bound kernel, so that costs nothing.  Scales multiply the group's fp32 sum:
// the weights are second operand, so a lane's results all belong to one weight row and
// it needs one scale per group.
#include "dense_common.h"

namespace ft {

using namespace dev;

namespace {

template <bool H>
struct Bias16 {
  // 16.0 and the place of its mantissa's 4 highest bits, in both halves of a word
  static constexpr uint32_t one = H ? 0x4c004c00u : 0x41804180u;
  static constexpr int sh = H ? 6 : 3;
  static constexpr uint32_t mask = 0x000f000fu << sh;
};

// Codes (0, 4), (1, 5), (2, 6), (3, 7) of a word of 8 as pairs of 16 + code.
template <bool H>
__device__ __forceinline__ i32x4_t widen(uint32_t v) {
  using B = Bias16<H>;
  auto at = [&](int i) -> int {
    const int s = B::sh - 4 * i;
    return (int)(((s >= 0 ? v << s : v >> -s) & B::mask) | B::one);
  };
  return i32x4_t{at(0), at(1), at(2), at(3)};
}
// 8 elements of x in the order of widen's.
__device__ __forceinline__ i32x4_t reorder(i32x4_t x) {
  const uint32_t a = x.x, b = x.y, c = x.z, d = x.w;
  return i32x4_t{(int)__builtin_amdgcn_perm(c, a, 0x05040100u), (int)__builtin_amdgcn_perm(c, a, 0x07060302u),
                 (int)__builtin_amdgcn_perm(d, b, 0x05040100u), (int)__builtin_amdgcn_perm(d, b, 0x07060302u)};
}

template <bool GU, bool H, int G, int NT, int W>
__global__ __launch_bounds__(64 * W) void w4_kernel(W4Args p) {
  constexpr int RB = GU ? 8 : 16, NG = 128 / G, PER = 4 / NG, U = NT == 1 ? 2 : 1;
  __shared__ float red[W][NT * 16][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * RB, t0 = blockIdx.y * (16 * NT);
  const int KG = p.K / G;
  const bool second = GU && n >= 8;
  const int64_t row = min(r0 + (GU ? (n & 7) : n), p.N - 1);
  const uint8_t* cp = (second ? p.codes2 : p.codes) + row * (p.K >> 1);
  const uint16_t* sp = (second ? p.scales2 : p.scales) + row * KG;
  const uint8_t* zp = second ? p.zeros2 : p.zeros;
  const bool hasz = zp != nullptr;
  zp += row * KG;
  const uint16_t* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xp[i] = p.x + (int64_t)min(t0 + i * 16 + n, p.T - 1) * p.ldx;
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{};
  const int chunks = (p.K + 127) >> 7;
  for (int c0 = wave; c0 < chunks; c0 += W * U) {
    uint4 q[U];
    i32x4_t fx[U][4][NT];
    float sc[U][NG];
    uint32_t zb[U][NG];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int k0 = (c0 + v * W) << 7;
      const int kc = k0 + g * 32;  // K % 32 == 0
      q[v] = *reinterpret_cast<const uint4*>(cp + (kc < p.K ? kc >> 1 : 0));
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int gi = min(k0 / G + j, KG - 1);
        sc[v][j] = to_f32<H>(sp[gi]);
        zb[v][j] = hasz ? zp[gi] : 8;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * 32 + g * 8;
        const bool ok = k < p.K;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          fx[v][j][i] = *reinterpret_cast<const i32x4_t*>(xp[i] + (ok ? k : 0));
          if (!ok) fx[v][j][i] = i32x4_t{};
        }
      }
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int k0 = (c0 + v * W) << 7;
      uint32_t w[4] = {q[v].x, q[v].y, q[v].z, q[v].w};
      // word j of row group g to row group j, word g
      auto s32 = [](uint32_t& a, uint32_t& b) {
        const u32x2_t r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        a = r.x;
        b = r.y;
      };
      auto s16 = [](uint32_t& a, uint32_t& b) {
        const u32x2_t r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
        a = r.x;
        b = r.y;
      };
      s32(w[0], w[2]);
      s32(w[1], w[3]);
      s16(w[0], w[1]);
      s16(w[2], w[3]);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        if (k0 + j * G >= p.K) break;
        const int bw = (int)((zb[v][j] << Bias16<H>::sh) * 0x10001u | Bias16<H>::one | 0x80008000u);
        const i32x4_t bias = {bw, bw, bw, bw};
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          f32x4_t s = f32x4_t{};
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const int jj = j * PER + e;
            const i32x4_t xr = reorder(fx[v][jj][i]);
            s = mfma16<H>(xr, widen<H>(w[jj]), s);
            s = mfma16<H>(xr, bias, s);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(sc[v][j], s[r], acc[i][r]);
        }
      }
    }
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
      p.h[(int64_t)tt * p.N + nn] = (uint16_t)pack2<H>(act_f(s, p.act) * u, 0.0f);
    } else if (p.y_f32) {
      if (p.res) s += static_cast<const float*>(p.res)[(int64_t)tt * p.ldr + nn];
      static_cast<float*>(p.y)[(int64_t)tt * p.ldy + nn] = s;
    } else {
      if (p.res) s += to_f32<H>(static_cast<const uint16_t*>(p.res)[(int64_t)tt * p.ldr + nn]);
      static_cast<uint16_t*>(p.y)[(int64_t)tt * p.ldy + nn] = (uint16_t)pack2<H>(s, 0.0f);
    }
  }
}

template <bool GU, bool H, int G>
int w4_go(const W4Args& A, hipStream_t s) {
  constexpr int RB = GU ? 8 : 16;
  const unsigned nb = (unsigned)(((int64_t)A.N + RB - 1) / RB);
  if (A.T <= 16)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 1, 8>), dim3(nb, 1), dim3(512), 0, s, A);
  else if (A.T <= 32)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 2, 8>), dim3(nb, 1), dim3(512), 0, s, A);
  else
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 4, 8>), dim3(nb, (unsigned)((A.T + 63) / 64)), dim3(512), 0, s, A);
  return launched("w4_kernel");
}
template <bool GU, bool H>
int w4_group(const W4Args& A, hipStream_t s) {
  if (A.G == 32) return w4_go<GU, H, 32>(A, s);
  if (A.G == 64) return w4_go<GU, H, 64>(A, s);
  return w4_go<GU, H, 128>(A, s);
}

}  // namespace

int launch_w4(const W4Args& A, bool gate_up, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((int64_t)(A.T + 63) / 64 > 65535) return fail(FT_EINVAL, "w4: more than 4194240 tokens");
  if (gate_up) return A.half ? w4_group<true, true>(A, s) : w4_group<true, false>(A, s);
  return A.half ? w4_group<false, true>(A, s) : w4_group<false, false>(A, s);
}

}  // namespace ft

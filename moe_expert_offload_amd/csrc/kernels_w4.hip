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

// Codes (0, 4), (1, 5), (2, 6), (3, 7) of a word of 8 as pairs of 16 + code: a shift and an and-or
// each.  `one` comes in a vector register and `mask` in a scalar one (an instruction reads at
// most one scalar operand and takes no second constant; written plainly it is an and and an or).
// Multiplying a byte into place, which keeps the codes in order, is slower: the 24-bit multiply
// runs at a quarter of the rate (the gate/up product of one token, d = 4096, d_ff = 11008: 24.0
// against 19.4 us).
template <bool H>
__device__ __forceinline__ i32x4_t widen(uint32_t v, uint32_t mask, uint32_t one) {
  auto at = [&](int i) -> int {
    const int s = Bias16<H>::sh - 4 * i;
    return (int)(((s >= 0 ? v << s : v >> -s) & mask) | one);
  };
  return i32x4_t{at(0), at(1), at(2), at(3)};
}
// 8 elements of x in the order of widen's.
__device__ __forceinline__ i32x4_t reorder(i32x4_t x) {
  const uint32_t a = x.x, b = x.y, c = x.z, d = x.w;
  return i32x4_t{(int)__builtin_amdgcn_perm(c, a, 0x05040100u), (int)__builtin_amdgcn_perm(c, a, 0x07060302u),
                 (int)__builtin_amdgcn_perm(d, b, 0x05040100u), (int)__builtin_amdgcn_perm(d, b, 0x07060302u)};
}

// Copies `bytes` (more than 0) from memory of any alignment to LDS, 16 at a time: a last short piece is moved
// back to end with the rest.  Less than one piece goes byte by byte.
__device__ __forceinline__ void stage_bytes(uint8_t* dst, const uint8_t* src, int bytes) {
  if (bytes >= 16) {
    for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16) {
      const int at = min(i, bytes - 16);
      uint4 v;
      __builtin_memcpy(&v, src + at, 16);
      __builtin_memcpy(dst + at, &v, 16);
    }
  } else if ((int)threadIdx.x < bytes) {
    dst[threadIdx.x] = src[threadIdx.x];
  }
}

// TK: tokens the kernel is made for (1, 4, 8: x in LDS, reordered once; 16, 32, 64 a pass: a chunk's x
// comes with its codes).  The tile's scales and zeros lie in LDS: loaded chunk by chunk each of these loads
// touches 16 rows and costs the load unit as much as the codes themselves; so do four loads of x that
// all rows of tokens share.  SL = false reads them from memory one by one, for K / group too
// large for LDS.  U chunks of a wave are in flight at once.
template <bool GU, bool H, int G, int TK, int W, int U, bool SL>
__global__ __launch_bounds__(64 * W, W / 4) void w4_kernel(W4Args p) {
  constexpr bool XL = TK <= 8;
  constexpr int RB = GU ? 8 : 16, NM = GU ? 2 : 1, NG = 128 / G, PER = 4 / NG, NT = TK < 16 ? 1 : TK / 16;
  constexpr int NR = TK == 1 ? 1 : 4;  // results of a lane that can belong to a token
  __shared__ float red[W][NT * 16][16];
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * RB, t0 = blockIdx.y * (16 * NT), nt = min(p.T - t0, 16 * NT);
  const int KG = p.K / G, KB = p.K >> 1;
  const int chunks = (p.K + 127) >> 7;
  const int nr = min(RB, p.N - r0), rl = min(GU ? (n & 7) : n, nr - 1);  // rows of the tile, the lane's
  const bool second = GU && n >= 8;
  const uint8_t* const cp = (second ? p.codes2 : p.codes) + (int64_t)(r0 + rl) * KB + g * 16;
  const bool hasz = (second ? p.zeros2 : p.zeros) != nullptr;
  uint32_t mask, one;
  asm("s_mov_b32 %0, %1" : "=s"(mask) : "i"(Bias16<H>::mask));
  asm("v_mov_b32 %0, %1" : "=v"(one) : "i"(Bias16<H>::one));

  // dynamic LDS: x [TK][K + 8] (XL), then the scales of the rows of each matrix, then their zeros
  const int xs = (p.K >> 3) + 1;  // row stride of x, pieces of 16 bytes: an odd number of them (K % 32 == 0)
  uint4* const sx = reinterpret_cast<uint4*>(dyn);
  uint8_t* const ss = dyn + (XL ? (size_t)min(p.T, TK) * xs * 16 : 0);
  uint8_t* const sz = ss + 16 * KG * 2;

  auto load = [&](uint4& q, int ci) {
    const int k0 = min(ci, chunks - 1) << 7;
    // K % 32 == 0: a lane's 32 codes are there or not as a whole
    q = *reinterpret_cast<const uint4*>(cp + (k0 + g * 32 < p.K ? k0 >> 1 : -g * 16));
  };

  uint4 q[U];
  if constexpr (XL) {
    const int per = p.K >> 3;
    i32x4_t v[TK];
    int c = threadIdx.x;
#pragma unroll
    for (int t = 0; t < TK; ++t)
      v[t] = *reinterpret_cast<const i32x4_t*>(p.x + (int64_t)min(t, nt - 1) * p.ldx + min(c, per - 1) * 8);
    while (true) {
      if (c < per) {
#pragma unroll
        for (int t = 0; t < TK; ++t)
          if (t < nt) {
            const i32x4_t r = reorder(v[t]);
            sx[t * xs + c] = make_uint4(r.x, r.y, r.z, r.w);
          }
      }
      c += 64 * W;
      if (c - (int)threadIdx.x >= per) break;
#pragma unroll
      for (int t = 0; t < TK; ++t)
        v[t] = *reinterpret_cast<const i32x4_t*>(p.x + (int64_t)min(t, nt - 1) * p.ldx + min(c, per - 1) * 8);
    }
  }
  if constexpr (SL) {
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const uint8_t* s = reinterpret_cast<const uint8_t*>(m ? p.scales2 : p.scales);
      const uint8_t* z = m ? p.zeros2 : p.zeros;
      stage_bytes(ss + m * 8 * KG * 2, s + (int64_t)r0 * KG * 2, nr * KG * 2);
      if (z) stage_bytes(sz + m * 8 * KG, z + (int64_t)r0 * KG, nr * KG);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) load(q[u], wave + u * W);
  const uint8_t* xp[NT];  // rows of x past T repeat the last one; their sums are dropped
  if constexpr (!XL) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
      xp[i] = reinterpret_cast<const uint8_t*>(p.x + (int64_t)(t0 + min(i * 16 + n, nt - 1)) * p.ldx) + g * 16;
  }
  const uint4* const xl = sx + min(n, nt - 1) * xs + g;
  const int lr = (second ? 8 : 0) + rl;
  const uint16_t* const sp = SL ? reinterpret_cast<const uint16_t*>(ss) + lr * KG
                                : (second ? p.scales2 : p.scales) + (int64_t)(r0 + rl) * KG;
  const uint8_t* const zp = SL ? sz + lr * KG : (second ? p.zeros2 : p.zeros) + (int64_t)(r0 + rl) * KG;
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{};
  if constexpr (XL || SL) __syncthreads();

  auto use = [&](const uint4& qu, const i32x4_t (&xu)[XL ? 1 : 4][NT], int k0) {
    uint32_t w[4] = {qu.x, qu.y, qu.z, qu.w};
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
      if (k0 + j * G >= p.K) break;  // a group is there whole or not at all
      const float scale = to_f32<H>(sp[k0 / G + j]);
      const uint32_t zb = hasz ? zp[k0 / G + j] : 8;
      const int bw = (int)((zb << Bias16<H>::sh) * 0x10001u | Bias16<H>::one | 0x80008000u);
      const i32x4_t bias = {bw, bw, bw, bw};
      f32x4_t s[NT];
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const i32x4_t wv = widen<H>(w[j * PER + e], mask, one);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const i32x4_t xr = XL ? *reinterpret_cast<const i32x4_t*>(xl + (k0 >> 3) + (j * PER + e) * 4)
                                : reorder(xu[XL ? 0 : j * PER + e][i]);
          s[i] = mfma16<H>(xr, wv, e ? s[i] : f32x4_t{});
          s[i] = mfma16<H>(xr, bias, s[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[i][r] = fmaf(scale, s[i][r], acc[i][r]);
    }
  };
  i32x4_t x[U][XL ? 1 : 4][NT];
  auto load_x = [&](i32x4_t (&xu)[XL ? 1 : 4][NT], int ci) {
    if constexpr (!XL) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k0 = min(ci, chunks - 1) << 7, k = k0 + j * 32 < p.K ? k0 + j * 32 : 0;
#pragma unroll
        for (int i = 0; i < NT; ++i) xu[j][i] = *reinterpret_cast<const i32x4_t*>(xp[i] + k * 2);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load_x(x[u], wave + u * W);
  __builtin_amdgcn_sched_barrier(0);
  int c0 = wave;
  for (; c0 + W * U < chunks; c0 += W * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      use(q[u], x[u], (c0 + u * W) << 7);  // all before the last chunk
      load(q[u], c0 + (U + u) * W);
      load_x(x[u], c0 + (U + u) * W);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + u * W < chunks) use(q[u], x[u], (c0 + u * W) << 7);
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) red[wave][i * 16 + g * 4 + r][n] = acc[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < nt * RB; e += 64 * W) {
    const int t = e / RB, c = e % RB;
    const int nn = r0 + c;
    if (c >= nr) continue;
    const int64_t tt = t0 + t;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][t][c];
    if constexpr (GU) {
      float u = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) u += red[w][t][c + 8];
      p.h[tt * p.N + nn] = (uint16_t)pack2<H>(act_f(s, p.act) * u, 0.0f);
    } else if (p.y_f32) {
      if (p.res) s += static_cast<const float*>(p.res)[tt * p.ldr + nn];
      static_cast<float*>(p.y)[tt * p.ldy + nn] = s;
    } else {
      if (p.res) s += to_f32<H>(static_cast<const uint16_t*>(p.res)[tt * p.ldr + nn]);
      static_cast<uint16_t*>(p.y)[tt * p.ldy + nn] = (uint16_t)pack2<H>(s, 0.0f);
    }
  }
}

template <bool GU, bool H, int G>
int w4_go(const W4Args& A, hipStream_t s) {
  constexpr int RB = GU ? 8 : 16;
  const unsigned tiles = (unsigned)(((int64_t)A.N + RB - 1) / RB), passes = (unsigned)((A.T + 63) / 64);
  const size_t sl = 16 * (size_t)(A.K / G) * 3;                                            // scales and zeros
  const size_t xl = (size_t)(A.T < 8 ? A.T : 8) * (2 * (size_t)A.K + 16), most = 128 << 10;  // 32 KB for the waves' parts
  if (sl > most)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 64, 8, 1, false>), dim3(tiles, passes), dim3(512), 0, s, A);
  else if (A.T == 1 && sl + xl <= most)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 1, 8, 4, true>), dim3(tiles), dim3(512), sl + xl, s, A);
  else if (A.T <= 4 && sl + xl <= most)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 4, 8, 4, true>), dim3(tiles), dim3(512), sl + xl, s, A);
  else if (A.T <= 8 && sl + xl <= most)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 8, 8, 4, true>), dim3(tiles), dim3(512), sl + xl, s, A);
  else if (A.T <= 16)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 16, 8, 4, true>), dim3(tiles), dim3(512), sl, s, A);
  else if (A.T <= 32)
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 32, 8, 2, true>), dim3(tiles), dim3(512), sl, s, A);
  else
    hipLaunchKernelGGL((w4_kernel<GU, H, G, 64, 8, 1, true>), dim3(tiles, passes), dim3(512), sl, s, A);
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

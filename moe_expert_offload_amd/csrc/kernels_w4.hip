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
// it needs one scale per group.  The price: an infinite x gives infinity - infinity, NaN, where the definition has
// an infinity (or NaN, for a weight of 0).
//
// A gate/up product's h is rounded to the activations' type, as the next product's MFMA operand.
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

// The scales and zeros of a tile's rows on their way from memory of any alignment to LDS, 16 bytes a
// thread at a time; a region's last short piece is moved back to end with the rest (regions have 16
// bytes or more).  All regions' loads leave before the first is written, without a branch between
// (one behind the other they took 1.7 us each).
template <int R>
struct Regions {
  const uint8_t* src[R];
  uint8_t* dst[R];  // 8-byte aligned, and so are the pieces: regions are multiples of 8 bytes
  int bytes[R];
  i32x4_t v[R];
  __device__ __forceinline__ void load(int i) {
    struct __attribute__((packed)) Any {
      i32x4_t v;
    };
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = reinterpret_cast<const Any*>(src[r] + min(i, bytes[r] - 16))->v;
  }
  __device__ __forceinline__ void store(int i) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i < bytes[r]) {
        uint2* d = reinterpret_cast<uint2*>(dst[r] + min(i, bytes[r] - 16));
        d[0] = make_uint2((uint32_t)v[r].x, (uint32_t)v[r].y);
        d[1] = make_uint2((uint32_t)v[r].z, (uint32_t)v[r].w);
      }
  }
};

// TK: tokens the kernel is made for.  Up to 16 (NX > 0): a chunk's x comes as whole rows of 256
// bytes, 4 tokens a load, and goes to its fragments through a piece of LDS of the wave's own, reordered on the way
// (a wave's LDS operations run in order, so that takes no barrier).  Loading fragments from
// memory takes 4 loads of 16 rows whatever the number of tokens, each as dear to the load unit as the
// chunk's codes.  32 and 64 a pass: fragments from memory.
// The tile's scales and zeros lie in LDS for the same reason: chunk by chunk each of these loads touches 16
// rows.  SL = false reads them from memory one by one, for K / group too large for LDS or matrices too small
// for Regions.
// U chunks of a wave are in flight at once; a chunk's registers are loaded again as it is used up.
template <bool GU, bool H, int G, int TK, int W, int U, bool SL>
__global__ __launch_bounds__(64 * W, W / 4) void w4_kernel(W4Args p) {
  constexpr int NX = TK > 16 ? 0 : (TK + 3) / 4;
  constexpr int RB = GU ? 8 : 16, NM = GU ? 2 : 1, NG = 128 / G, PER = 4 / NG, NT = TK <= 16 ? 1 : TK / 16;
  constexpr int NR = TK == 1 ? 1 : 4;  // results of a lane that can belong to a token
  constexpr int XS = 17;               // row stride of x in LDS, in 16 bytes: rows start on different banks
  __shared__ float red[W][NT * 16][16];
  __shared__ uint4 sx[W][NX ? NX * 4 * XS : 1];
  extern __shared__ __attribute__((aligned(16))) uint8_t ss[];  // scales of the tile's rows, then zeros
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * RB, t0 = blockIdx.y * (16 * NT), nt = min(p.T - t0, 16 * NT);
  const int KG = p.K / G, KB = p.K >> 1;
  const int chunks = (p.K + 127) >> 7;
  const int nr = min(RB, p.N - r0), rl = min(GU ? (n & 7) : n, nr - 1);  // rows of the tile, the lane's
  const int rb = SL ? min(r0, p.N - RB) : r0;  // LDS holds RB rows from here
  const bool second = GU && n >= 8;
  const uint8_t* const cp = (second ? p.codes2 : p.codes) + (int64_t)(r0 + rl) * KB + g * 16;
  const bool hasz = (second ? p.zeros2 : p.zeros) != nullptr;
  uint32_t mask, one;
  asm("s_mov_b32 %0, %1" : "=s"(mask) : "i"(Bias16<H>::mask));
  asm("v_mov_b32 %0, %1" : "=v"(one) : "i"(Bias16<H>::one));
  uint8_t* const sz = ss + 16 * KG * 2;

  // rows of x past T repeat the last one; their sums are dropped
  const uint8_t* xp[NX ? NX : NT];
#pragma unroll
  for (int i = 0; i < (NX ? NX : NT); ++i) {
    const int t = NX ? i * 4 + g : i * 16 + n;
    xp[i] = reinterpret_cast<const uint8_t*>(p.x + (int64_t)(t0 + min(t, nt - 1)) * p.ldx) + (NX ? n : g) * 16;
  }
  struct Chunk {
    uint4 q;
    i32x4_t x[NX ? NX : 4 * NT];
  };
  Chunk ch[U];
  auto load = [&](Chunk& c, int ci) {
    const int k0 = min(ci, chunks - 1) << 7;  // past the last: that one again, not used
    // K % 32 == 0: a lane's 32 codes are there or not as a whole; what is not there is not used
    c.q = *reinterpret_cast<const uint4*>(cp + (k0 + g * 32 < p.K ? k0 >> 1 : -g * 16));
    if constexpr (NX > 0) {
      const int k = k0 + n * 8 < p.K ? k0 * 2 : -n * 16;
#pragma unroll
      for (int i = 0; i < NX; ++i) c.x[i] = *reinterpret_cast<const i32x4_t*>(xp[i] + k);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * 32 < p.K ? k0 + j * 32 : 0;
#pragma unroll
        for (int i = 0; i < NT; ++i) c.x[j * NT + i] = *reinterpret_cast<const i32x4_t*>(xp[i] + k * 2);
      }
    }
  };
  Regions<2 * NM> rg;
  const int at = threadIdx.x * 16;
  if constexpr (SL) {
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const uint8_t *sc = reinterpret_cast<const uint8_t*>(m ? p.scales2 : p.scales), *z = m ? p.zeros2 : p.zeros;
      rg.src[m] = sc + (int64_t)rb * KG * 2;
      rg.dst[m] = ss + m * 8 * KG * 2;
      rg.bytes[m] = RB * KG * 2;
      rg.src[NM + m] = (z ? z : sc) + (int64_t)rb * KG;  // without zeros these bytes are not used
      rg.dst[NM + m] = sz + m * 8 * KG;
      rg.bytes[NM + m] = RB * KG;
    }
    rg.load(at);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) load(ch[u], wave + u * W);
  if constexpr (SL) {
    rg.store(at);
    for (int i = at + 64 * W * 16; i - at < RB * KG * 2; i += 64 * W * 16) {
      rg.load(i);
      rg.store(i);
    }
    __syncthreads();
  }
  const int lr = (second ? 8 : 0) + rl + r0 - rb;
  const uint16_t* const sp = SL ? reinterpret_cast<const uint16_t*>(ss) + lr * KG
                                : (second ? p.scales2 : p.scales) + (int64_t)(r0 + rl) * KG;
  const uint8_t* const zp = SL      ? sz + lr * KG
                            : hasz ? (second ? p.zeros2 : p.zeros) + (int64_t)(r0 + rl) * KG
                                   : reinterpret_cast<const uint8_t*>(sp);  // read, not used
  f32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4_t{};

  uint4* const xw = sx[wave] + g * XS + n;
  const uint4* const xr = sx[wave] + min(n, NX * 4 - 1) * XS + g;
  auto use = [&](const Chunk& c, int k0) {
    if constexpr (NX > 0) {
#pragma unroll
      for (int i = 0; i < NX; ++i) xw[i * 4 * XS] = __builtin_bit_cast(uint4, reorder(c.x[i]));
      __builtin_amdgcn_wave_barrier();
    }
    uint32_t w[4] = {c.q.x, c.q.y, c.q.z, c.q.w};
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
    float scales[NG];
    uint32_t zeros[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int gi = NG == 1 ? k0 / G : min(k0 / G + j, KG - 1);
      scales[j] = to_f32<H>(sp[gi]);
      zeros[j] = zp[gi];
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      if (k0 + j * G >= p.K) break;  // a group is there whole or not at all
      const float scale = scales[j];
      const uint32_t zb = hasz ? zeros[j] : 8;
      const int bw = (int)((zb << Bias16<H>::sh) * 0x10001u | Bias16<H>::one | 0x80008000u);
      const i32x4_t bias = {bw, bw, bw, bw};
      f32x4_t s[NT];
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int jj = j * PER + e;
        const i32x4_t wv = widen<H>(w[jj], mask, one);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          i32x4_t xv;
          if constexpr (NX > 0)
            xv = __builtin_bit_cast(i32x4_t, xr[jj * 4]);
          else
            xv = reorder(c.x[jj * NT + i]);
          s[i] = mfma16<H>(xv, wv, e ? s[i] : f32x4_t{});
          s[i] = mfma16<H>(xv, bias, s[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[i][r] = fmaf(scale, s[i][r], acc[i][r]);
    }
    if constexpr (NX > 0) __builtin_amdgcn_wave_barrier();
  };
  __builtin_amdgcn_sched_barrier(0);
  int c0 = wave;
  for (; c0 + W * U < chunks; c0 += W * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      use(ch[u], (c0 + u * W) << 7);  // all before the last chunk
      load(ch[u], c0 + (U + u) * W);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + u * W < chunks) use(ch[u], (c0 + u * W) << 7);
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
  const size_t sl = 16 * (size_t)(A.K / G) * 3;  // scales and zeros
  auto go = [&](auto kernel, unsigned y, size_t lds) { hipLaunchKernelGGL(kernel, dim3(tiles, y), dim3(512), lds, s, A); };
  // Chunks in flight a wave: more of them is longer code, which these short kernels wait for as it is
  // fetched (one token d = 4096, d_ff = 11008, group 128, chunks in flight 1, 2, 3, 4, 8: 21.4, 20.6, 23.9, 22.2,
  // 31.3 us; 16 tokens d = 4096, d_ff = 2048, group 32, 1, 2, 3: 14.9, 15.2, 16.1 us).
  if (sl > (64 << 10) || A.N < RB || RB * (A.K / G) < 16)
    go(w4_kernel<GU, H, G, 64, 8, 1, false>, passes, 0);
  else if (A.T == 1)
    go(w4_kernel<GU, H, G, 1, 8, 2, true>, 1, sl);
  else if (A.T <= 4)
    go(w4_kernel<GU, H, G, 4, 8, 2, true>, 1, sl);
  else if (A.T <= 8)
    go(w4_kernel<GU, H, G, 8, 8, 2, true>, 1, sl);
  else if (A.T <= 16)
    go(w4_kernel<GU, H, G, 16, 8, 1, true>, 1, sl);
  else if (A.T <= 32)
    go(w4_kernel<GU, H, G, 32, 8, 2, true>, 1, sl);
  else
    go(w4_kernel<GU, H, G, 64, 8, 1, true>, passes, sl);
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
  if (A.T > 65535 * 64) return fail(FT_EINVAL, "w4: more than 4194240 tokens");
  if (gate_up) return A.half ? w4_group<true, true>(A, s) : w4_group<true, false>(A, s);
  return A.half ? w4_group<false, true>(A, s) : w4_group<false, false>(A, s);
}

}  // namespace ft

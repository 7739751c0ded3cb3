// Products in 8-bit integers with a scale for each token and each channel, and the gated block on
// them.  gfx950 only.
//
//   s[t] = max|x[t]| / 127, q[t, k] = round(x[t, k] / s[t])
//   y[t, n] = (sum over k of q[t, k] c[n, k]) * scale[n] * s[t] (+ residual)
//   block: h = act(a) * u rounded to the activations' type, quantised as x is, then the down product
//
// The sums are whole numbers in 32 bits, exact in any order (K <= 65536: at most 2^30 in magnitude); the two scales
// and the residual are applied in fp32.  h is rounded to 16 bits on its way to its codes: its row's
// largest element is known only when all of its product's tiles are done, so h goes through
// memory, and half the bytes cost less than 1/127 of the largest does.
#include <type_traits>

#include "dense_cut.h"
#include "i8_common.h"

namespace ft {

using namespace dev;

namespace {

// ---- rows to codes ------------------------------------------------------------------
// ROWT threads a row (quant_row).
template <bool H, int ROWT, int NP>
__global__ __launch_bounds__(ROWT) void i8_quant_kernel(const uint16_t* src, int64_t ld, int rows, int n, int8_t* codes,
                                                        float* scales) {
  __shared__ uint32_t red[ROWT / 64];
  const int64_t row = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (row >= rows) return;  // the whole block
  quant_row<H, ROWT, NP>(src + row * ld, n, codes + row * n, scales + row, red);
}

// ---- products -------------------------------------------------------------------------

enum {
  kOut,    // y (+ residual) in 16 bits or fp32
  kGateUp  // two matrices side by side, h = act(a) * u in 16 bits
};

struct I8Args {
  const int8_t *a, *b, *b2;  // codes of the tokens [M, K], of the channels [N, K]; b2: up
  const uint16_t* x16;       // the tokens in 16 bits instead, quantised by each block
  const float *ta, *sb, *sb2;  // scales of the tokens and of the channels
  int64_t lda;
  int M, N, K, act;
  void* c;
  int64_t ldc;
  int c_f32, wide;  // wide: rows of c and residual may be accessed 16 bytes at a time
  const void* res;
  int64_t ldr;
  uint16_t* h;  // kGateUp: [M, N]
  // how tiles are shared: see I8Cut
  int tiles_m, tiles_n, whole, blocks, per, parts;
  int* part;  // sums of pieces
};

template <bool H>
__device__ __forceinline__ void store1(const I8Args& p, int64_t m, int n, float v) {
  if (p.c_f32) {
    if (p.res) v += static_cast<const float*>(p.res)[m * p.ldr + n];
    static_cast<float*>(p.c)[m * p.ldc + n] = v;
  } else {
    if (p.res) v += to_f32<H>(static_cast<const uint16_t*>(p.res)[m * p.ldr + n]);
    static_cast<uint16_t*>(p.c)[m * p.ldc + n] = (uint16_t)pack2<H>(v, 0.0f);
  }
}

// ---- few rows: the weights stream once --------------------------------------------------
// A block owns 16 channels (kGateUp: 8 of each matrix), its waves take chunks of 256 k in turn and add their sums in
// LDS.  v_mfma_i32_16x16x64: the weights are the second operand, so each byte is loaded once, straight into
// registers; tokens past the last repeat it and their sums are dropped.
//
// Tokens' codes as fragments from memory would touch 16 rows a load, as dear to the load unit as the weights'. So
//   QX            x comes in 16 bits and each block quantises it for itself, whole, into LDS, while its first
//                 weights are on their way (i8_own_codes)
//   TK up to 16   a chunk's codes come as whole rows of 256 bytes, 4 tokens a load, and go to their fragments through
//                 a piece of LDS of the wave's own (a wave's LDS operations run in order: no barrier)
//   32, 64        fragments from memory
// One chunk a wave, loaded again as it is used up: two or more take registers that further waves use better (45 MB of
// weights, 2 tokens: K = 4096 11.6 us, with two chunks 13.0, with four 14.3).
template <int MODE, bool H, bool QX, int TK, int W>
__global__ __launch_bounds__(64 * W, W == 8 ? 6 : 4) void i8_skinny_kernel(I8Args p) {
  constexpr bool GU = MODE == kGateUp;
  constexpr int RB = GU ? 8 : 16, NT = TK <= 16 ? 1 : TK / 16;
  constexpr int NX = QX || TK > 16 ? 0 : (TK + 3) / 4;
  constexpr int XS = 17;  // row stride of a chunk's codes in LDS, in 16 bytes: rows start on different banks
  __shared__ int red[W][NT * 16][16];
  __shared__ uint4 sx[W][NX ? NX * 4 * XS : 1];
  __shared__ uint32_t top[W];
  __shared__ float own_scale[16];
  extern __shared__ uint4 own[];  // QX: codes, rows of K + 16 bytes
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * RB;
  const int row = r0 + (GU ? (n & 7) : n);
  const int8_t* wp = (GU && n >= 8 ? p.b2 : p.b) + (int64_t)min(row, p.N - 1) * p.K;
  const int chunks = (p.K + 255) >> 8;
  const int8_t* xp[NX ? NX : NT];
  if constexpr (!QX) {
#pragma unroll
    for (int i = 0; i < (NX ? NX : NT); ++i)
      xp[i] = p.a + (int64_t)min(NX ? i * 4 + g : i * 16 + n, p.M - 1) * p.lda;
  }
  struct Chunk {
    i32x4_t w[4];
    i32x4_t x[QX ? 1 : NX ? NX : 4 * NT];
  };
  Chunk ch;
  auto load = [&](Chunk& c, int ci) {
    const int k0 = ci << 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j * 64 + g * 16;  // K % 16 == 0
      c.w[j] = *reinterpret_cast<const i32x4_t*>(wp + (k < p.K ? k : 0));
      if (k >= p.K) c.w[j] = i32x4_t{};
    }
    if constexpr (NX > 0) {
      const int k = k0 + n * 16;
#pragma unroll
      for (int i = 0; i < NX; ++i) c.x[i] = *reinterpret_cast<const i32x4_t*>(xp[i] + (k < p.K ? k : 0));
    } else if constexpr (!QX) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * 64 + g * 16;
#pragma unroll
        for (int i = 0; i < NT; ++i) c.x[j * NT + i] = *reinterpret_cast<const i32x4_t*>(xp[i] + (k < p.K ? k : 0));
      }
    }
  };
  if (wave < chunks) load(ch, wave);

  const int own_row = p.K + 16;  // bytes
  if constexpr (QX) {
    // W / (T to a power of two) waves a row (none left over: T <= W); a thread holds at most NP pieces of 8
    constexpr int NP = kOwnCodes / 8 / (64 * W);
    int per = W;
    while (per > 1 && W / per < p.M) per >>= 1;
    const int t = wave / per, first = wave - wave % per, at = (wave % per) * 64 + lane, pieces = p.K >> 3;
    uint4 v[NP];
    uint32_t m = 0;
    const uint4* src = reinterpret_cast<const uint4*>(p.x16 + (int64_t)min(t, p.M - 1) * p.lda);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int q = at + i * per * 64;
      v[i] = q < pieces ? src[q] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) m = amax4(v[i], m);
    m = wave_umax(m);
    if (lane == 0) top[wave] = m;
    __syncthreads();
    for (int w = 0; w < per; ++w) m = max(m, top[first + w]);
    if (t < p.M) {
      const RowScale r = row_scale<H>(m);
      uint2* d = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(own) + t * own_row);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int q = at + i * per * 64;
        const uint32_t e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        if (q < pieces) d[q] = row_codes8<H>(e, r);
      }
      if (wave == first && lane == 0) own_scale[t] = r.scale;
    }
    __syncthreads();
  }

  i32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = i32x4_t{};
  uint4* const xw = sx[wave] + g * XS + n;
  const uint4* const xr = sx[wave] + min(n, NX * 4 - 1) * XS + g;
  const uint8_t* const xo = reinterpret_cast<const uint8_t*>(own) + min(n, p.M - 1) * own_row;
  auto use = [&](const Chunk& c, int ci) {
    if constexpr (NX > 0) {
#pragma unroll
      for (int i = 0; i < NX; ++i) xw[i * 4 * XS] = __builtin_bit_cast(uint4, c.x[i]);
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        i32x4_t x;
        if constexpr (QX)
          x = *reinterpret_cast<const i32x4_t*>(xo + min((ci << 8) + j * 64 + g * 16, p.K));  // past K: weights 0
        else if constexpr (NX > 0)
          x = __builtin_bit_cast(i32x4_t, xr[j * 4]);
        else
          x = c.x[j * NT + i];
        acc[i] = mfma16(x, c.w[j], acc[i]);
      }
    if constexpr (NX > 0) __builtin_amdgcn_wave_barrier();
  };
  __builtin_amdgcn_sched_barrier(0);
  for (int c = wave; c < chunks; c += W) {
    use(ch, c);
    if (c + W < chunks) load(ch, c + W);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][i * 16 + g * 4 + r][n] = acc[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 16 * RB; e += 64 * W) {
    const int t = e / RB, c = e % RB, nn = r0 + c;
    if (t >= p.M || nn >= p.N) continue;
    const float ts = QX ? own_scale[t] : p.ta[t];
    int s = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][t][c];
    if constexpr (GU) {
      int u = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) u += red[w][t][c + 8];
      const float v = act_f(i8_value(s, p.sb[nn], ts), p.act) * i8_value(u, p.sb2[nn], ts);
      p.h[(int64_t)t * p.N + nn] = (uint16_t)pack2<H>(v, 0.0f);
    } else {
      store1<H>(p, t, nn, i8_value(s, p.sb[nn], ts));
    }
  }
}

// ---- many rows: tiles -------------------------------------------------------------------
// A tile's scales: of its BM tokens, then of its BN channels (kGateUp: BN / 2 of gate, then of up); those past
// the ends are not used.  Read in the epilogue from LDS: from memory, each group of four waited for its
// own round trip (8192 x 4096 x 4096: 172 us, so 124 us).
template <int MODE, int BM, int BN, int THREADS>
__device__ __forceinline__ void stage_scales(const I8Args& p, float* s, int m0, int n0) {
  for (int i = threadIdx.x; i < BM + BN; i += THREADS) {
    float v;
    if (i < BM) {
      v = p.ta[min(m0 + i, p.M - 1)];
    } else if (MODE == kGateUp) {
      const int c = i - BM;
      v = c < BN / 2 ? p.sb[min(n0 + c, p.N - 1)] : p.sb2[min(n0 + c - BN / 2, p.N - 1)];
    } else {
      v = p.sb[min(n0 + i - BM, p.N - 1)];
    }
    s[i] = v;
  }
}

// The same by one load of each wave straight into LDS, so that nobody waits for it by itself.
template <int MODE, int BM, int BN>
__device__ __forceinline__ void load_scales(const I8Args& p, uint32_t lds, int m0, int n0, int wave, int lane) {
  const int i = wave * 64;
  const float* src;
  int left;
  if (i < BM) {
    src = p.ta + m0 + i;
    left = p.M - m0 - i;
  } else if (i < BM + BN) {
    const int c = i - BM;
    const bool up = MODE == kGateUp && c >= BN / 2;
    const int n = n0 + (up ? c - BN / 2 : c);
    src = (up ? p.sb2 : p.sb) + n;
    left = p.N - n;
  } else {
    return;
  }
  lds_load4(rsrc_of(src), lane < left ? (uint32_t)lane * 4 : kOOB, 0, lds + i * 4);
}

// What becomes of one 32-row piece of a wave's sums: c0 and c1 are its 32x32 results at channels n0 + b0 and
// n0 + b1 (kGateUp: gate and up of the same ones).  The lane holds row `r` of the tile, and in quad q the
// channels 8 q + 4 hi + 0..3 of each.  scales: the tile's, of BM tokens first.  QH >= 0: quads 2 QH and 2 QH + 1 alone.
template <int MODE, bool H, int BM, int BN, int QH = -1>
__device__ __forceinline__ void i8_epilogue(const I8Args& p, const i32x16_t& c0, const i32x16_t& c1, const float* scales,
                                            int m0, int r, int n0, int b0, int b1, int hi) {
  const int m = m0 + r;
  const bool mok = m < p.M;
  const float ts = scales[r];
  const float4* cs = reinterpret_cast<const float4*>(scales + BM);
  if constexpr (MODE == kGateUp) {
#pragma unroll
    for (int q = QH > 0 ? 2 : 0; q < (QH == 0 ? 2 : 4); q += 2) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = (b0 + 8 * (q + e) + 4 * hi) >> 2, k = 4 * (q + e);
        const float4 sg = cs[c], su = cs[c + BN / 8];
        const float h0 = act_f(i8_value(c0[k], sg.x, ts), p.act) * i8_value(c1[k], su.x, ts);
        const float h1 = act_f(i8_value(c0[k + 1], sg.y, ts), p.act) * i8_value(c1[k + 1], su.y, ts);
        const float h2 = act_f(i8_value(c0[k + 2], sg.z, ts), p.act) * i8_value(c1[k + 2], su.z, ts);
        const float h3 = act_f(i8_value(c0[k + 3], sg.w, ts), p.act) * i8_value(c1[k + 3], su.w, ts);
        w[2 * e] = pack2<H>(h0, h1);
        w[2 * e + 1] = pack2<H>(h2, h3);
      }
      swap_halves(w[0], w[2]);
      swap_halves(w[1], w[3]);
      const int n = n0 + b0 + 8 * q + 8 * hi;  // N % 16 == 0
      if (mok && n < p.N) *reinterpret_cast<uint4*>(p.h + (int64_t)m * p.N + n) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    // The residual's pieces leave together, from addresses inside it (those past its ends are not used): one behind the
    // other each waited for its own round trip (the block of 8192 tokens with a residual, d = 4096, d_ff = 2048: 241 us, so 235).
    // (Rows through LDS in pieces of 512 bytes instead of 32 took 267: the whole block waits at each pass.)
    constexpr int Q0 = QH > 0 ? 2 : 0, Q1 = QH == 0 ? 2 : 4;
    uint4 old[2][2];
    const bool wide16 = p.wide && !p.c_f32 && p.res;
    if (wide16) {
      const uint16_t* r = static_cast<const uint16_t*>(p.res) + (int64_t)min(m, p.M - 1) * p.ldr;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = Q0; q < Q1; q += 2)
          old[j][q >> 1] = *reinterpret_cast<const uint4*>(r + min(n0 + (j ? b1 : b0) + 8 * q + 8 * hi, p.N - 8));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int b = j ? b1 : b0;
      const i32x16_t& c = j ? c1 : c0;
#pragma unroll
      for (int q = Q0; q < Q1; q += 2) {
        float v[8];  // after the exchange: channels b + 8 (q + hi) .. + 7
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 sc = cs[(b + 8 * (q + e) + 4 * hi) >> 2];
          const int k = 4 * (q + e);
          v[4 * e] = i8_value(c[k], sc.x, ts);
          v[4 * e + 1] = i8_value(c[k + 1], sc.y, ts);
          v[4 * e + 2] = i8_value(c[k + 2], sc.z, ts);
          v[4 * e + 3] = i8_value(c[k + 3], sc.w, ts);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t x = __float_as_uint(v[e]), y = __float_as_uint(v[4 + e]);
          swap_halves(x, y);
          v[e] = __uint_as_float(x);
          v[4 + e] = __uint_as_float(y);
        }
        const int n = n0 + b + 8 * q + 8 * hi;
        const bool ok = mok && n < p.N;
        if (!p.wide) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (mok && n + e < p.N) store1<H>(p, m, n + e, v[e]);
        } else if (p.c_f32) {  // wide: N % 8 == 0
          if (ok) {
            float* o = static_cast<float*>(p.c) + (int64_t)m * p.ldc + n;
            if (p.res) {
              const float* r = static_cast<const float*>(p.res) + (int64_t)m * p.ldr + n;
              const float4 a = *reinterpret_cast<const float4*>(r), b = *reinterpret_cast<const float4*>(r + 4);
              v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
              v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
            }
            *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        } else {
          if (wide16) {
            const uint4 r = old[j][q >> 1];
            const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[2 * e] += lo16<H>(rw[e]);
              v[2 * e + 1] += hi16<H>(rw[e]);
            }
          }
          if (ok)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c) + (int64_t)m * p.ldc + n) =
                make_uint4(pack2<H>(v[0], v[1]), pack2<H>(v[2], v[3]), pack2<H>(v[4], v[5]), pack2<H>(v[6], v[7]));
        }
      }
    }
  }
}

// Tile index to its place: consecutive tiles walk 8 tile rows per column of tiles.
struct TilePos {
  int m, n;
};
__device__ __forceinline__ TilePos tile_pos(const I8Args& p, int t) {
  const int per = 8 * p.tiles_n, grp = t / per, first = grp * 8;
  const int rows = min(8, p.tiles_m - first), in = t - grp * per;
  return {first + in % rows, in / rows};
}

// A block's work: a whole tile, or (slot >= 0) one of the `blocks` pieces of a tile behind those.  Consecutive ones share
// an XCD.
struct Piece {
  int tile, s_begin, s_end, slot;
};
__device__ __forceinline__ Piece piece_of(const I8Args& p, int stages) {
  if ((int)blockIdx.x < p.whole) return {xcd_logical_block(blockIdx.x, p.whole), 0, stages, -1};
  const int b = xcd_logical_block(blockIdx.x - p.whole, p.parts), t = b / p.blocks, s = (b - t * p.blocks) * p.per;
  return {p.whole + t, s, min(stages, s + p.per), b};
}

// Two 32x32 sums of a wave among a piece's: 2048 whole numbers, quads of 4 channels by lane.
__device__ __forceinline__ void store_part(int* at, const i32x16_t (&c)[2], int lane) {
  i32x4_t* d = reinterpret_cast<i32x4_t*>(at) + lane;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) d[(j * 4 + q) * 64] = i32x4_t{c[j][4 * q], c[j][4 * q + 1], c[j][4 * q + 2], c[j][4 * q + 3]};
}
// The sums of `n` pieces, `stride` numbers apart: quads 2 QH and 2 QH + 1 of both results, four pieces' loads at once.
template <int QH>
__device__ __forceinline__ void sum_parts(i32x16_t (&c)[2], const int* at, size_t stride, int n, int lane) {
  c[0] = c[1] = i32x16_t{};
  for (int b0 = 0; b0 < n; b0 += 4) {
    i32x4_t v[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const i32x4_t* d = reinterpret_cast<const i32x4_t*>(at + (size_t)min(b0 + b, n - 1) * stride) + lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[b][e] = d[((e >> 1) * 4 + 2 * QH + (e & 1)) * 64];
    }
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (b0 + b < n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[e >> 1][4 * (2 * QH + (e & 1)) + i] += v[b][e][i];
  }
}

// The places of operands in LDS, the walk over k and the cut into shared tiles are those of the 16-bit
// products (kernels_dense.hip, gemm_kernel and gemm256_kernel, for operands along k): an LDS row is 128 bytes,
// here 128 k, and an MFMA of 32 k takes the cycles of one of 16 there, so the same bytes are
// loaded and read in the same time for twice the operations.

// BM x 128 tiles, BM 128 or 64: 4 waves of BM / 2 x 64, both operands straight into one of S LDS buffers, S - 1 stages
// ahead.  Loads past the last stage are masked (they write zeros nobody reads), which keeps the count of the wait.
template <int MODE, bool H, int BM, int S>
__global__ __launch_bounds__(256, 1) void i8_tile128_kernel(I8Args p) {
  constexpr bool GU = MODE == kGateUp;
  constexpr int MT = BM / 64, ABYTES = BM * 128, SBYTES = ABYTES + 16384;
  constexpr int LA = BM / 32, LB = 4;  // 1 KB loads a wave issues a stage
  extern __shared__ __attribute__((aligned(1024))) uint8_t sm[];  // S * SBYTES
  __shared__ __attribute__((aligned(16))) float scales[BM + 128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, hi = lane >> 5, l31 = lane & 31;
  const int stages = (p.K + 127) >> 7;
  const Piece w = piece_of(p, stages);
  const int s_begin = w.s_begin, s_end = w.s_end;
  const TilePos tp = tile_pos(p, w.tile);
  const int m0 = tp.m * BM, n0 = tp.n * (GU ? 64 : 128);

  uint32_t offA[LA], offB[LB];
  int kA[LA], kB[LB];  // first k of the piece within the stage
#pragma unroll
  for (int j = 0; j < LA; ++j) {
    const int r = (wave * LA + j) * 8 + (lane >> 3), pc = (lane & 7) ^ ((r >> 1) & 7);
    kA[j] = pc * 16;
    offA[j] = m0 + r < p.M ? (uint32_t)(r * p.lda + pc * 16) : kOOB;
  }
#pragma unroll
  for (int j = 0; j < LB; ++j) {
    const int r = (wave * LB + j) * 8 + (lane >> 3), pc = (lane & 7) ^ ((r >> 1) & 7);
    const int n = GU ? (r >> 6) * 32 + (r & 31) : r;  // blocks of 32 rows alternate between gate and up
    kB[j] = pc * 16;
    offB[j] = n0 + n < p.N ? (uint32_t)(n * p.K + pc * 16) : kOOB;
  }
  const uint32_t sm0 = lds_addr(sm);
  auto load_stage = [&](int s, int place) {
    const int k0 = s << 7, left = s < s_end ? p.K - k0 : 0;
    const uint32_t dst = sm0 + place * SBYTES;
    const auto ra = rsrc_of(p.a + m0 * p.lda + k0);
#pragma unroll
    for (int j = 0; j < LA; ++j) lds_load16(ra, kA[j] < left ? offA[j] : kOOB, 0, dst + (wave * LA + j) * 1024);
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int8_t* w = GU && ((wave * LB + j) & 4) ? p.b2 : p.b;
      lds_load16(rsrc_of(w + (int64_t)n0 * p.K + k0), kB[j] < left ? offB[j] : kOOB, 0, dst + ABYTES + (wave * LB + j) * 1024);
    }
  };
  auto frag = [&](const uint8_t* base, int row, int slice) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(base + (row + l31) * 128 + (((2 * slice + hi) ^ ((l31 >> 1) & 7)) << 4));
  };
  i32x16_t acc[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = i32x16_t{};
  load_scales<MODE, BM, 128>(p, lds_addr(scales), m0, n0, wave, lane);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) load_stage(s_begin + i, i);
  int here = 0;
  for (int s = s_begin; s < s_end; ++s) {
    // this wave's loads of stage s have landed; past the barrier everyone's have, and nobody
    // reads the buffer before it any more
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 2) * (LA + LB)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    load_stage(s + S - 1, here == 0 ? S - 1 : here - 1);
    const uint8_t *sa = sm + here * SBYTES, *sb = sa + ABYTES;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      i32x4_t fa[MT], fb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[j] = frag(sb, wn * 64 + j * 32, k);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i] = frag(sa, wm * (BM / 2) + i * 32, k);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(fb[j], fa[i], acc[i][j]);
    }
    // the reads above are done before anyone passes the next barrier
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    here = here == S - 1 ? 0 : here + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the masked loads too: LDS is another block's afterwards
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (w.slot >= 0) {
      store_part(p.part + (size_t)w.slot * (BM * 128) + (wave * MT + i) * 2048, acc[i], lane);
    } else {
      const int b = wn * (GU ? 32 : 64);
      i8_epilogue<MODE, H, BM, 128>(p, acc[i][0], acc[i][1], scales, m0, wm * (BM / 2) + i * 32 + l31, n0, b, b + 32, hi);
    }
  }
}

// The shared tiles of the kernel above: a block per tile, 32-row piece of the waves and half of their quads.
template <int MODE, bool H, int BM>
__global__ __launch_bounds__(256) void i8_join128_kernel(I8Args p) {
  constexpr int MT = BM / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, t = blockIdx.x / (2 * MT), i = (blockIdx.x >> 1) % MT;
  __shared__ __attribute__((aligned(16))) float scales[BM + 128];
  const TilePos tp = tile_pos(p, p.whole + t);
  const int m0 = tp.m * BM, n0 = tp.n * (MODE == kGateUp ? 64 : 128), r = wm * (BM / 2) + i * 32;
  stage_scales<MODE, BM, 128, 256>(p, scales, m0, n0);
  __syncthreads();
  if (m0 + r >= p.M) return;
  const int* at = p.part + (size_t)t * p.blocks * (BM * 128) + (wave * MT + i) * 2048;
  const int c = wn * (MODE == kGateUp ? 32 : 64);
  auto half = [&](auto h) {
    constexpr int QH = decltype(h)::value;
    i32x16_t acc[2];
    sum_parts<QH>(acc, at, BM * 128, p.blocks, lane);
    i8_epilogue<MODE, H, BM, 128, QH>(p, acc[0], acc[1], scales, m0, r + (lane & 31), n0, c, c + 32, lane >> 5);
  };
  if (blockIdx.x & 1)
    half(std::integral_constant<int, 1>{});
  else
    half(std::integral_constant<int, 0>{});
}

// 128 MH x 256 tiles, 8 waves, each 64 rows and 32 channels of every 128 x 128 quarter.  A stage is regions of
// 16 KB (A0, B0, B1 and with MH = 2 A1); the waves 4..7 run one section behind the waves 0..3, so on every
// SIMD one wave multiplies while the other reads.  Sections of a stage for the first group:
//   MH = 2 (two stages in LDS)   read A0, B0, B1 of s; load A1 of s + 1; wait for A1 of s
//                                A0 x B0, A0 x B1
//                                read A1 of s; load A0, B0, B1 of s + 2; wait for A0, B0, B1 of s + 1
//                                A1 x B1, A1 x B0
//   MH = 1 (three stages)        read A0, B0, B1 of s; load those of s + 2; wait for those of s + 1
//                                A0 x B0, A0 x B1
// Every section ends with a barrier.  A region is loaded again two sections after the first group read it, one
// after the second did (both end a read section with their reads done), and is waited for by both groups
// at least one barrier before its first read.  Loads past the last stage are masked (they write
// zeros nobody reads), which keeps the counts of the waits.
template <int MODE, bool H, int MH>
__global__ __launch_bounds__(512, 2) void i8_tile256_kernel(I8Args p) {
  constexpr bool GU = MODE == kGateUp;
  constexpr int REG = 16384;
  enum { A0 = 0, B0 = REG, B1 = 2 * REG, A1 = 3 * REG, STAGE = (2 + MH) * REG, PLACES = MH == 2 ? 2 : 3 };
  __shared__ __attribute__((aligned(1024))) uint8_t sm[PLACES * STAGE];
  constexpr int BM = 128 * MH, PART = BM * 256;  // rows of a tile, numbers of its sums
  __shared__ __attribute__((aligned(16))) float scales[BM + 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, hi = lane >> 5, l31 = lane & 31;
  const int stages = (p.K + 127) >> 7;

  const Piece w = piece_of(p, stages);
  const int s_begin = w.s_begin, s_end = w.s_end;
  const TilePos tp = tile_pos(p, w.tile);
  const int m0 = tp.m * BM, n0 = tp.n * (GU ? 128 : 256);
  // rows of a wave in the two halves: those past the end are neither read nor multiplied
  const bool any[2] = {m0 + wm * 64 < p.M, m0 + 128 + wm * 64 < p.M};

  // ---- loads: a wave brings chunks 2 wave and 2 wave + 1 (1 KB) of every region ----
  uint32_t offA[MH][2], offB[2][2];  // [half][chunk]
  int kq[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = (wave * 2 + j) * 8 + (lane >> 3), pk = (lane & 7) ^ ((r >> 1) & 7);
    kq[j] = pk * 16;
#pragma unroll
    for (int h = 0; h < MH; ++h) offA[h][j] = m0 + h * 128 + r < p.M ? (uint32_t)(r * p.lda + pk * 16) : kOOB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int nh = n0 + (GU ? 0 : h * 128);
      offB[h][j] = nh + r < p.N ? (uint32_t)(r * p.K + pk * 16) : kOOB;
    }
  }
  // Each region's source moves on by a stage per load.
  const uint32_t sm0 = lds_addr(sm) + wave * 2048;
  const int k0 = s_begin << 7;
  const int8_t* pa[2] = {p.a + m0 * p.lda + k0, p.a + (m0 + 128) * p.lda + k0};
  const int8_t* pb[2] = {p.b + (int64_t)n0 * p.K + k0, (GU ? p.b2 + (int64_t)n0 * p.K : p.b + (int64_t)(n0 + 128) * p.K) + k0};
  auto load = [&](int s, const int8_t*& src, const uint32_t (&off)[2], uint32_t region, int place) {
    const int left = s < s_end ? p.K - (s << 7) : 0;
    const auto rs = rsrc_of(src);
#pragma unroll
    for (int j = 0; j < 2; ++j) lds_load16(rs, kq[j] < left ? off[j] : kOOB, 0, sm0 + place * STAGE + region + j * 1024);
    src += 128;
  };
  auto load_a = [&](int s, int h, int place) { load(s, pa[h], offA[h], h ? A1 : A0, place); };
  auto load_b = [&](int s, int h, int place) { load(s, pb[h], offB[h], h ? B1 : B0, place); };

  // ---- fragments of a region: 32 rows from `row`, slice of 32 k ----
  auto frag = [&](const uint8_t* base, int row, int slice) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(base + (row + l31) * 128 + (((2 * slice + hi) ^ ((l31 >> 1) & 7)) << 4));
  };
  i32x16_t acc[2 * MH][2];  // [2 half + 32-row piece][half of the channels]
#pragma unroll
  for (int i = 0; i < 2 * MH; ++i) acc[i][0] = acc[i][1] = i32x16_t{};
  i32x4_t fa[2][4], fb0[4], fb1[4];
  auto read_a = [&](const uint8_t* base) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i][k] = frag(base, wm * 64 + i * 32, k);
  };
  auto read_b = [&](const uint8_t* base, i32x4_t (&f)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = frag(base, wn * 32, k);
  };
  auto multiply = [&](int half) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[2 * half + i][0] = mfma32(fb0[k], fa[i][k], acc[2 * half + i][0]);
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[2 * half + i][1] = mfma32(fb1[k], fa[i][k], acc[2 * half + i][1]);
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
    load_scales<MODE, BM, 256>(p, lds_addr(scales), m0, n0, wave, lane);  // the oldest: waited for with the first stage
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
    // RAGGED: the tile has rows past the end.
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
    const int m = m0 + (i >> 1) * 128 + wm * 64 + (i & 1) * 32;
    if (w.slot >= 0) {
      if (m < p.M) store_part(p.part + (size_t)w.slot * PART + (wave * 2 * MH + i) * 2048, acc[i], lane);
    } else {
      i8_epilogue<MODE, H, BM, 256>(p, acc[i][0], acc[i][1], scales, m0, m - m0 + l31, n0, wn * 32, wn * 32 + 128, hi);
    }
  }
}

// The tiles whose stages several blocks shared: a block per tile, 32-row piece of the waves and half of their quads;
// bound by memory.
template <int MODE, bool H, int MH>
__global__ __launch_bounds__(512) void i8_join256_kernel(I8Args p) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, i = (blockIdx.x >> 1) % (2 * MH), t = blockIdx.x / (4 * MH);
  const TilePos tp = tile_pos(p, p.whole + t);
  __shared__ __attribute__((aligned(16))) float scales[MH * 128 + 256];
  const int m0 = tp.m * 128 * MH, n0 = tp.n * (MODE == kGateUp ? 128 : 256), r = (i >> 1) * 128 + wm * 64 + (i & 1) * 32;
  stage_scales<MODE, MH * 128, 256, 512>(p, scales, m0, n0);
  __syncthreads();
  if (m0 + r >= p.M) return;
  constexpr int PART = MH * 128 * 256;
  const int* at = p.part + (size_t)t * p.blocks * PART + (wave * 2 * MH + i) * 2048;
  auto half = [&](auto h) {
    constexpr int QH = decltype(h)::value;
    i32x16_t acc[2];
    sum_parts<QH>(acc, at, PART, p.blocks, lane);
    i8_epilogue<MODE, H, MH * 128, 256, QH>(p, acc[0], acc[1], scales, m0, r + (lane & 31), n0, wn * 32, wn * 32 + 128, lane >> 5);
  };
  if (blockIdx.x & 1)
    half(std::integral_constant<int, 1>{});
  else
    half(std::integral_constant<int, 0>{});
}

// ---- launches -------------------------------------------------------------------------

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int MODE, bool H>
int i8_go(I8Args& A, hipStream_t s) {
  const I8Cut c = i8_cut_of(A.M, MODE == kGateUp ? 2 * (int64_t)A.N : A.N, A.K);
  if (c.tile == 0) {
    constexpr int RB = MODE == kGateUp ? 8 : 16;
    const unsigned nb = (unsigned)((A.N + RB - 1) / RB);
    // 16 waves a block where there are few blocks (one token, K = N = 4096: 7.6 us, with 8 waves 9.0), else 8 (K = 4096,
    // N = 11008: 13.1, with 16 waves 20.5)
    const bool few = nb < 2 * kUnits;
    auto go = [&](auto wide, auto slim, size_t lds) {
      if (few)
        hipLaunchKernelGGL(wide, dim3(nb), dim3(1024), lds, s, A);
      else
        hipLaunchKernelGGL(slim, dim3(nb), dim3(512), lds, s, A);
    };
    if (A.x16)
      go(i8_skinny_kernel<MODE, H, true, 16, 16>, i8_skinny_kernel<MODE, H, true, 16, 8>, (size_t)A.M * (A.K + 16) + 16);
    else if (A.M <= 4)
      go(i8_skinny_kernel<MODE, H, false, 4, 16>, i8_skinny_kernel<MODE, H, false, 4, 8>, 0);
    else if (A.M <= 16)
      go(i8_skinny_kernel<MODE, H, false, 16, 16>, i8_skinny_kernel<MODE, H, false, 16, 8>, 0);
    else if (A.M <= 32)
      hipLaunchKernelGGL((i8_skinny_kernel<MODE, H, false, 32, 16>), dim3(nb), dim3(1024), 0, s, A);
    else
      hipLaunchKernelGGL((i8_skinny_kernel<MODE, H, false, 64, 16>), dim3(nb), dim3(1024), 0, s, A);
    return launched("i8_skinny_kernel");
  }
  const size_t es = A.c_f32 ? 4 : 2;
  A.wide = A.N % 8 == 0 && aligned(A.c, 16) && aligned(A.res, 16) && A.ldc * es % 16 == 0 && (!A.res || A.ldr * es % 16 == 0);
  A.tiles_m = c.tiles_m;
  A.tiles_n = c.tiles_n;
  A.whole = c.whole;
  A.blocks = c.blocks;
  A.per = c.per;
  A.parts = c.parts;
  if (c.tile == 256) {
    hipLaunchKernelGGL((i8_tile256_kernel<MODE, H, 2>), dim3((unsigned)(c.whole + c.parts)), dim3(512), 0, s, A);
    if (c.rest) hipLaunchKernelGGL((i8_join256_kernel<MODE, H, 2>), dim3((unsigned)c.rest * 8), dim3(512), 0, s, A);
  } else if (c.tile == 384) {
    hipLaunchKernelGGL((i8_tile256_kernel<MODE, H, 1>), dim3((unsigned)(c.whole + c.parts)), dim3(512), 0, s, A);
    if (c.rest) hipLaunchKernelGGL((i8_join256_kernel<MODE, H, 1>), dim3((unsigned)c.rest * 4), dim3(512), 0, s, A);
  } else {
    auto go = [&](auto tile, size_t stage, int deep, auto join, unsigned pieces) {
      hipLaunchKernelGGL(tile, dim3((unsigned)(c.whole + c.parts)), dim3(256), deep * stage, s, A);
      if (c.rest) hipLaunchKernelGGL(join, dim3((unsigned)c.rest * pieces), dim3(256), 0, s, A);
    };
    if (c.tile == 64)
      go(i8_tile128_kernel<MODE, H, 64, 3>, 24576, 3, i8_join128_kernel<MODE, H, 64>, 2);
    else if (c.deep)
      go(i8_tile128_kernel<MODE, H, 128, 3>, 32768, 3, i8_join128_kernel<MODE, H, 128>, 4);
    else
      go(i8_tile128_kernel<MODE, H, 128, 2>, 32768, 2, i8_join128_kernel<MODE, H, 128>, 4);
  }
  return launched("i8_tile_kernel");
}

template <int MODE>
int i8_product(I8Args& A, bool half, hipStream_t s) {
  return half ? i8_go<MODE, true>(A, s) : i8_go<MODE, false>(A, s);
}

void fill_out(I8Args& A, const I8Out& o) {
  A.c = o.y;
  A.ldc = o.ldy;
  A.c_f32 = o.f32;
  A.res = o.res;
  A.ldr = o.ldr;
}

}  // namespace

int launch_i8_quant(const uint16_t* src, int64_t ld, int rows, int n, bool half, int8_t* codes, float* scales, void* stream) {
  if (rows <= 0) return FT_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto go = [&](auto kernel, int threads) {
    // a grid's first dimension holds fewer than 2^32 threads
    const unsigned b = (unsigned)rows, x = b < 65536 ? b : 65536;
    hipLaunchKernelGGL(kernel, dim3(x, (b + x - 1) / x), dim3(threads), 0, s, src, ld, rows, n, codes, scales);
  };
  // few long rows: more threads on each, so that none reads its row twice
  const bool few = rows <= 2 * kUnits && n > 4096;
  if (half)
    few ? go(i8_quant_kernel<true, 1024, 2>, 1024) : go(i8_quant_kernel<true, 256, 2>, 256);
  else
    few ? go(i8_quant_kernel<false, 1024, 2>, 1024) : go(i8_quant_kernel<false, 256, 2>, 256);
  return launched("i8_quant_kernel");
}

int launch_i8_gemm(const I8Rows& x, const I8Mat& w, const I8Out& o, bool half, int* part, void* stream) {
  if (x.T <= 0) return FT_OK;
  I8Args A{};
  A.a = x.codes;
  A.x16 = x.x16;
  A.lda = x.ld;
  A.ta = x.scales;
  A.b = w.codes;
  A.sb = w.scales;
  A.M = x.T;
  A.N = w.N;
  A.K = w.K;
  A.part = part;
  fill_out(A, o);
  return i8_product<kOut>(A, half, static_cast<hipStream_t>(stream));
}

int launch_i8_gate_up(const I8Rows& x, const I8Mat& gate, const I8Mat& up, int act, uint16_t* h, bool half, int* part,
                      void* stream) {
  if (x.T <= 0) return FT_OK;
  I8Args A{};
  A.a = x.codes;
  A.x16 = x.x16;
  A.lda = x.ld;
  A.ta = x.scales;
  A.b = gate.codes;
  A.b2 = up.codes;
  A.sb = gate.scales;
  A.sb2 = up.scales;
  A.M = x.T;
  A.N = gate.N;
  A.K = gate.K;
  A.act = act;
  A.h = h;
  A.part = part;
  return i8_product<kGateUp>(A, half, static_cast<hipStream_t>(stream));
}

}  // namespace ft

// Products in 8-bit integers with a scale for each token and each channel, and the gated block on
// them.  gfx950 only.
//
//   s[t] = max|x[t]| / 127, q[t, k] = round(x[t, k] / s[t])
//   y[t, n] = (sum over k of q[t, k] c[n, k]) * scale[n] * s[t] (+ residual)
//   block: h = act(a) * u rounded to the activations' type, quantised as x is, then the down product
//
// The sums are whole numbers in 32 bits, exact in any order (K <= 65536: below 2^30); the two scales
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
// A row is held in registers between its largest element and its codes, NP pieces of 8 elements a
// thread; rows longer than that are read again.  ROWT threads a row.
template <bool H, int ROWT, int NP>
__global__ __launch_bounds__(256) void i8_quant_kernel(const uint16_t* src, int64_t ld, int rows, int n, int8_t* codes,
                                                       float* scales) {
  __shared__ uint32_t red[4];
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (256 / ROWT) + threadIdx.x / ROWT;
  if (row >= rows) return;  // ROWT = 256: the whole block; else whole waves
  const int at = threadIdx.x % ROWT, pieces = n >> 3;
  const uint4* q = reinterpret_cast<const uint4*>(src + row * ld);
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
    m = max(max(red[0], red[1]), max(red[2], red[3]));
  }
  const RowScale r = row_scale<H>(m);
  uint2* d = reinterpret_cast<uint2*>(codes + row * n);
  auto put = [&](int p, const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    d[p] = row_codes8<H>(w, r);
  };
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (at + i * ROWT < pieces) put(at + i * ROWT, v[i]);
  for (int p = at + NP * ROWT; p < pieces; p += ROWT) put(p, q[p]);
  if (at == 0) scales[row] = r.scale;
}

// ---- products -------------------------------------------------------------------------

enum {
  kOut,    // y (+ residual) in 16 bits or fp32
  kGateUp  // two matrices side by side, h = act(a) * u in 16 bits
};

struct I8Args {
  const int8_t *a, *b, *b2;  // codes of the tokens [M, K], of the channels [N, K]; b2: up
  const float *ta, *sb, *sb2;  // scales of the tokens and of the channels
  int64_t lda;
  int M, N, K, act;
  void* c;
  int64_t ldc;
  int c_f32, wide;  // wide: rows of c and residual may be accessed 16 bytes at a time
  const void* res;
  int64_t ldr;
  uint16_t* h;  // kGateUp: [M, N]
  // how tiles are shared: see Cut
  int tiles_m, tiles_n, whole, rest, group, blocks, per, parts;
  int* part;  // sums of pieces
};

// Four scales from n on; those past the end are not used.
__device__ __forceinline__ float4 scales4(const float* s, int n, int N) {
  struct __attribute__((packed, aligned(4))) Any {
    float4 v;
  };
  if (n + 4 <= N) return reinterpret_cast<const Any*>(s + n)->v;
  return make_float4(s[min(n, N - 1)], s[min(n + 1, N - 1)], s[min(n + 2, N - 1)], s[min(n + 3, N - 1)]);
}

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
// Up to 16 * NT tokens a pass.  A block owns 16 channels (kGateUp: 8 of each matrix), its waves split k
// in steps of 64 and add their sums in LDS.  v_mfma_i32_16x16x64: the weights are the second operand, so
// each byte is loaded once, straight into registers; tokens past the last repeat it and their
// sums are dropped.
template <int MODE, bool H, int NT, int W>
__global__ __launch_bounds__(64 * W) void i8_skinny_kernel(I8Args p) {
  constexpr bool GU = MODE == kGateUp;
  constexpr int RB = GU ? 8 : 16, U = NT <= 2 ? 4 : 2;
  __shared__ int red[W][NT * 16][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.x * RB, t0 = blockIdx.y * (16 * NT);
  const int row = r0 + (GU ? (n & 7) : n);
  const int8_t* wp = GU && n >= 8 ? p.b2 : p.b;
  wp += (int64_t)min(row, p.N - 1) * p.K;
  const int8_t* xp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) xp[i] = p.a + (int64_t)min(t0 + i * 16 + n, p.M - 1) * p.lda;
  i32x4_t acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = i32x4_t{};
  const int steps = (p.K + 63) >> 6;  // of 64 k; pairs of steps go to the waves in turn
  for (int s0 = 2 * wave; s0 < steps; s0 += 2 * W * (U / 2)) {
    i32x4_t fw[U], fx[U][NT];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int s = s0 + (v >> 1) * 2 * W + (v & 1);
      const int k = s * 64 + g * 16;
      const bool ok = k < p.K;  // K % 16 == 0
      const int ka = ok ? k : 0;
      fw[v] = *reinterpret_cast<const i32x4_t*>(wp + ka);
#pragma unroll
      for (int i = 0; i < NT; ++i) fx[v][i] = *reinterpret_cast<const i32x4_t*>(xp[i] + ka);
      if (!ok) fw[v] = i32x4_t{};
    }
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = mfma16(fx[v][i], fw[v], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][i * 16 + g * 4 + r][n] = acc[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < NT * 16 * RB; e += 64 * W) {
    const int t = e / RB, c = e % RB;
    const int tt = t0 + t, nn = r0 + c;
    if (tt >= p.M || nn >= p.N) continue;
    const float ts = p.ta[tt];
    int s = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][t][c];
    if constexpr (GU) {
      int u = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) u += red[w][t][c + 8];
      const float v = act_f(i8_value(s, p.sb[nn], ts), p.act) * i8_value(u, p.sb2[nn], ts);
      p.h[(int64_t)tt * p.N + nn] = (uint16_t)pack2<H>(v, 0.0f);
    } else {
      store1<H>(p, tt, nn, i8_value(s, p.sb[nn], ts));
    }
  }
}

// ---- launches -------------------------------------------------------------------------

template <int MODE, bool H>
int i8_go(I8Args& A, hipStream_t s) {
  constexpr int RB = MODE == kGateUp ? 8 : 16;
  const unsigned nb = (unsigned)((A.N + RB - 1) / RB);
  for (int t = 0; t < A.M; t += 64 * 65535) {
    I8Args P = A;
    P.M = A.M - t < 64 * 65535 ? A.M - t : 64 * 65535;
    P.a += t * A.lda;
    P.ta += t;
    P.c = P.c ? static_cast<uint8_t*>(P.c) + t * A.ldc * (A.c_f32 ? 4 : 2) : nullptr;
    P.res = P.res ? static_cast<const uint8_t*>(P.res) + t * A.ldr * (A.c_f32 ? 4 : 2) : nullptr;
    P.h = P.h ? P.h + (int64_t)t * A.N : nullptr;
    if (P.M <= 16)
      hipLaunchKernelGGL((i8_skinny_kernel<MODE, H, 1, 16>), dim3(nb, 1), dim3(1024), 0, s, P);
    else if (P.M <= 32)
      hipLaunchKernelGGL((i8_skinny_kernel<MODE, H, 2, 8>), dim3(nb, 1), dim3(512), 0, s, P);
    else
      hipLaunchKernelGGL((i8_skinny_kernel<MODE, H, 4, 8>), dim3(nb, (unsigned)((P.M + 63) / 64)), dim3(512), 0, s, P);
  }
  return launched("i8_skinny_kernel");
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
  auto go = [&](auto kernel, int per) {
    // a grid's first dimension holds fewer than 2^32 threads
    const unsigned b = ((unsigned)rows + per - 1) / per, x = b < 65536 ? b : 65536;
    hipLaunchKernelGGL(kernel, dim3(x, (b + x - 1) / x), dim3(256), 0, s, src, ld, rows, n, codes, scales);
  };
  if (half)
    go(i8_quant_kernel<true, 256, 2>, 1);
  else
    go(i8_quant_kernel<false, 256, 2>, 1);
  return launched("i8_quant_kernel");
}

int launch_i8_gemm(const I8Rows& x, const I8Mat& w, const I8Out& o, bool half, int* part, void* stream) {
  if (x.T <= 0) return FT_OK;
  I8Args A{};
  A.a = x.codes;
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

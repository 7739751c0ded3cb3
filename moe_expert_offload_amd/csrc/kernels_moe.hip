// A whole routed layer for a few tokens whose experts are all on the device.  gfx950 only.
//
//   logits = x W_r^T; the k largest of the allowed experts; gates = softmax over those
//   y[t] = sum over j of gates[t, j] * Wd_e (silu(Wg_e x[t]) * (Wu_e x[t])), e = idx[t, j] (+ residual[t])
//
// Launches: the logits; the experts' gate and up products; 8-bit records of more than a few pairs: h's codes; the down
// product.  More than 24 tokens: the top-k behind the logits.  The second does the top-k of every token otherwise, and groups
// the routed pairs by expert, every block by itself (in LDS; a layer of 64 tokens has 512 pairs at most), so
// that no launch and no wait across blocks lies between; the down product sums a token's experts where they leave
// it, so there is no combine.  (Both products in one launch, down's blocks waiting for the parts of h that they need:
// 77 us against 65 for one token, d = 4096, d_ff = 2048, top-6, bf16; a wait across XCDs costs more than a launch.)
//
// Both stream the routed experts' rows once, whatever number of tokens takes them: a wavefront holds a few rows in registers
// and applies each token of the expert to them (lane l takes the 16-byte pieces l, l + 64, ... of a row, 1 KB a load).
// Bound by memory: one token as above 64 us, 302 MB at 4.7 TB/s; 16 tokens in MXFP4 214 us, 5 TB/s.  From about 3
// tokens an expert on by the vector instructions that apply each: there the matrix instructions take over (below).
//
// Records (bf16, MXFP4) as in include/ft.h; MXFP4 weights are dequantised exactly and applied to the bf16
// x and the fp32 h.  8-bit records: x and h in 8 bits as ft_i8_quant gives them (h rounded to bf16 before),
// whole-number sums, as the blocks of kernels_i8.hip.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "i8_common.h"
#include "router_device.h"

namespace ft {

using namespace dev;

namespace {

constexpr int NT = 1024, NW = NT / 64;  // threads and wavefronts of a block, one block a compute unit

// The routed pairs by expert (of 512 pairs at most), as gate/up leaves them for down.
struct Grouped {
  int32_t groups;
  int32_t grp[FT_PLAN_CAP];      // a pair's group, -1: left out (no expert, or none of the given ones)
  int32_t slot[FT_PLAN_CAP];     // of a group
  int32_t off[FT_PLAN_CAP + 1];  // first of a group's pairs in `pair`
  int32_t pair[FT_PLAN_CAP];     // pairs by group
  float gate[FT_PLAN_CAP];
};
static_assert(sizeof(Grouped) <= kMoeGroupedBytes, "the workspace's share");

struct MoeArgs {
  const uint16_t* x;
  const float* logits;
  const uint8_t* allowed;
  const uint8_t* rec;
  const int32_t* slot_of;
  int T, d, f, E, k, n_slots;
  size_t S;
  int32_t* idx;
  float* gates;
  int ranked;  // both are there
  Grouped* grouped;
  void* xv;    // x as it is multiplied: bf16 x itself, MXFP4 in planes (the matrix form: x itself), 8-bit records codes (scales xs)
  float* xs;
  int8_t* hq;  // 8-bit records: h in 8 bits (scales hs)
  float* hs;
  void* h;  // [T k, f]: fp32 in planes, 8-bit records bf16
  int split;    // matrix form of down: blocks that share rows of y (moe_down_split), their sums in part [split, T, d]
  float* part;
  const void* res;
  void* y;
  int y_f32;
  int rows;     // down: rows of a block; gate/up's matrix form: tokens of a part
  int lds_vec;  // the tokens' rows (gate/up: x, down: h) are staged in LDS
};

// ---- 16-byte pieces of rows, by format --------------------------------------------------
// E elements a piece; gate/up multiplies it by NU 16-byte parts of x, down by ND parts of h.
template <int FMT>
struct Fmt;
template <>
struct Fmt<FT_W_BF16> {
  static constexpr int E = 8, NU = 1, ND = 2;
  typedef float Acc;
};
template <>
struct Fmt<FT_W_MXFP4> {
  static constexpr int E = 32, NU = 4, ND = 8;
  typedef float Acc;
};
template <>
struct Fmt<FT_W_I8> {
  static constexpr int E = 16, NU = 1, ND = 1;
  typedef int Acc;
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float dot_bf16(uint4 a, uint4 b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, x[i]), __builtin_bit_cast(bf16x2_t, y[i]), acc, false);
  return acc;
}
__device__ __forceinline__ float dot_f32(uint4 a, uint4 h0, uint4 h1, float acc) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  const uint32_t h[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(bf_lo(w[i]), __uint_as_float(h[2 * i]), acc);
    acc = fmaf(bf_hi(w[i]), __uint_as_float(h[2 * i + 1]), acc);
  }
  return acc;
}
// 2^(s - 127) for an E8M0 byte.
__device__ __forceinline__ float e8m0(uint32_t s) { return s ? __uint_as_float(s << 23) : 0x1p-127f; }
template <int B>
__device__ __forceinline__ bf16x2_t mx_pair(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, B);
}
template <int B>
__device__ __forceinline__ f32x2_t mx_pair32(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, B);
}
__device__ __forceinline__ float mx_word_bf16(uint32_t w, uint4 x, float acc) {
  acc = __builtin_amdgcn_fdot2_f32_bf16(mx_pair<0>(w), __builtin_bit_cast(bf16x2_t, x.x), acc, false);
  acc = __builtin_amdgcn_fdot2_f32_bf16(mx_pair<1>(w), __builtin_bit_cast(bf16x2_t, x.y), acc, false);
  acc = __builtin_amdgcn_fdot2_f32_bf16(mx_pair<2>(w), __builtin_bit_cast(bf16x2_t, x.z), acc, false);
  return __builtin_amdgcn_fdot2_f32_bf16(mx_pair<3>(w), __builtin_bit_cast(bf16x2_t, x.w), acc, false);
}
__device__ __forceinline__ float mx_word_f32(uint32_t w, uint4 a, uint4 b, float acc) {
  f32x2_t v = mx_pair32<0>(w);
  acc = fmaf(v.x, __uint_as_float(a.x), acc);
  acc = fmaf(v.y, __uint_as_float(a.y), acc);
  v = mx_pair32<1>(w);
  acc = fmaf(v.x, __uint_as_float(a.z), acc);
  acc = fmaf(v.y, __uint_as_float(a.w), acc);
  v = mx_pair32<2>(w);
  acc = fmaf(v.x, __uint_as_float(b.x), acc);
  acc = fmaf(v.y, __uint_as_float(b.y), acc);
  v = mx_pair32<3>(w);
  acc = fmaf(v.x, __uint_as_float(b.z), acc);
  return fmaf(v.y, __uint_as_float(b.w), acc);
}
__device__ __forceinline__ int dot_i8(uint4 a, uint4 b, int acc) {
  acc = __builtin_amdgcn_sdot4((int)a.x, (int)b.x, acc, false);
  acc = __builtin_amdgcn_sdot4((int)a.y, (int)b.y, acc, false);
  acc = __builtin_amdgcn_sdot4((int)a.z, (int)b.z, acc, false);
  return __builtin_amdgcn_sdot4((int)a.w, (int)b.w, acc, false);
}
// acc + piece w (MXFP4: under scale byte sc) times the parts v of x (DOWN: of h).
template <int FMT, bool DOWN, int NV>
__device__ __forceinline__ typename Fmt<FMT>::Acc piece_dot(uint4 w, uint32_t sc, const uint4 (&v)[NV],
                                                            typename Fmt<FMT>::Acc acc) {
  if constexpr (FMT == FT_W_I8) {
    return dot_i8(w, v[0], acc);
  } else if constexpr (FMT == FT_W_BF16) {
    if constexpr (DOWN)
      return dot_f32(w, v[0], v[1], acc);
    else
      return dot_bf16(w, v[0], acc);
  } else {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) s = DOWN ? mx_word_f32(c[q], v[2 * q], v[2 * q + 1], s) : mx_word_bf16(c[q], v[q], s);
    return fmaf(s, e8m0(sc), acc);
  }
}

// Sums over the wavefront of N values of each lane at once: halves of lanes that hold one value's parts take on
// another's.  The lane gets in v[0] the total of value total_of<N>(lane) (of 8: v[0] that of the first four,
// v[1] that of the last).
template <int N>
__device__ __forceinline__ int total_of(int lane) {
  return N == 1 ? 0 : N == 2 ? lane >> 5 : ((lane >> 4) & 1) * 2 + (lane >> 5);
}
template <int CTRL, class T>
__device__ __forceinline__ T dpp_of(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
template <class T>
__device__ __forceinline__ T row_total(T v) {  // over 16 lanes
  v += dpp_of<0xb1>(v);   // quad_perm [1,0,3,2]
  v += dpp_of<0x4e>(v);   // quad_perm [2,3,0,1]
  v += dpp_of<0x141>(v);  // row_half_mirror
  return v + dpp_of<0x140>(v);  // row_mirror
}
template <class T>
__device__ __forceinline__ T join32(T a, T b) {  // lanes 0..31: a's, 32..63: b's
  const u32x2_t r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = r.x, y = r.y;
  return __builtin_bit_cast(T, x) + __builtin_bit_cast(T, y);
}
template <class T>
__device__ __forceinline__ T join16(T a, T b) {  // rows 0 and 2: a's, 1 and 3: b's
  const u32x2_t r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
  const uint32_t x = r.x, y = r.y;
  return __builtin_bit_cast(T, x) + __builtin_bit_cast(T, y);
}
template <int N, class T>
__device__ __forceinline__ void wave_totals(T (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "");
  if constexpr (N == 1) {
    const T a = row_total(v[0]), h = join32(a, a);
    v[0] = join16(h, h);
  } else if constexpr (N == 2) {
    const T a = row_total(join32(v[0], v[1]));
    v[0] = join16(a, a);
  } else {
#pragma unroll
    for (int q = 0; q < N / 4; ++q)
      v[q] = row_total(join16(join32(v[4 * q], v[4 * q + 1]), join32(v[4 * q + 2], v[4 * q + 3])));
  }
}

// A record's parts (byte offsets).
struct Rec {
  uint32_t up, down, gs, us, ds;  // codes (the gate's at 0), scales
};
template <int FMT>
__device__ __forceinline__ Rec rec_of(int d, int f) {
  Rec r;
  const size_t n = (size_t)d * f;
  if constexpr (FMT == FT_W_BF16) {
    r = Rec{(uint32_t)(2 * n), (uint32_t)(4 * n), 0, 0, 0};
  } else if constexpr (FMT == FT_W_MXFP4) {
    const size_t c = n / 2, s = n / 32;
    r = Rec{(uint32_t)c, (uint32_t)(2 * c), (uint32_t)(3 * c), (uint32_t)(3 * c + s), (uint32_t)(3 * c + 2 * s)};
  } else {
    r = Rec{(uint32_t)n, (uint32_t)(2 * n), (uint32_t)(3 * n), (uint32_t)(3 * n + 4 * (size_t)f), (uint32_t)(3 * n + 8 * (size_t)f)};
  }
  return r;
}
template <int FMT>
__device__ __forceinline__ int row_bytes(int n) {
  return FMT == FT_W_BF16 ? 2 * n : FMT == FT_W_MXFP4 ? n / 2 : n;
}

// ---- the routed pairs by expert, in LDS ---------------------------------------------------
struct Plan : Grouped {
  int32_t id[FT_PLAN_CAP];  // expert of a pair
  int32_t first[FT_E_MAX];  // an expert's first pair, then its group
  unsigned long long tokens[FT_PLAN_CAP];  // a group's, a bit each: a token takes an expert once
  int32_t wave_sum[NW];
};

// Exclusive prefix sums over the block's threads of at most 16 bits' worth each; returns this thread's.
__device__ __forceinline__ int block_prefix(int v, int32_t* wave_sums, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int in = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(in, o, WAVE);
    if (lane >= o) in += t;
  }
  if (lane == 63) wave_sums[wave] = in;
  __syncthreads();
  int base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    base += w < wave ? wave_sums[w] : 0;
    total += wave_sums[w];
  }
  __syncthreads();
  return base + in - v;
}

// The record of a pair's expert, -1: none.
__device__ __forceinline__ int slot_of(const MoeArgs& p, int id) {
  if (id < 0 || id >= p.E) return -1;
  const int slot = p.slot_of ? p.slot_of[id] : id;
  return slot >= 0 && slot < p.n_slots ? slot : -1;
}

// Groups in the order of their first pair, pairs within a group in theirs (every block makes the same plan).  id and
// gate are set.  Up to 64 pairs, by one wavefront: a lane a pair.
__device__ void plan_of_a_wave(Plan& P, const MoeArgs& p, int lane) {
  const int n = p.T * p.k;
  const int id = lane < n ? P.id[lane] : -1, slot = slot_of(p, id);
  int before = 0, first_of = lane;
  for (int q = n - 1; q >= 0; --q) {
    const bool same = __builtin_amdgcn_readlane(id, q) == id;
    before += same && q < lane;
    if (same) first_of = q;
  }
  const unsigned long long firsts = __ballot(slot >= 0 && first_of == lane);
  const int groups = __popcll(firsts), grp = slot >= 0 ? __popcll(firsts & ((1ull << first_of) - 1)) : -1;
  int off = 0;  // pairs of the groups before this one
  for (int q = 0; q < n; ++q) {
    const int g = __builtin_amdgcn_readlane(grp, q);
    off += g >= 0 && g < grp;
  }
  if (lane < n) P.grp[lane] = grp;
  if (grp >= 0) {
    P.pair[off + before] = lane;
    if (first_of == lane) {
      P.slot[grp] = slot;
      P.off[grp] = off;
    }
  }
  const int all = __popcll(__ballot(grp >= 0));
  if (lane == 0) {
    P.groups = groups;
    P.off[groups] = all;
  }
}
// More pairs, by the block (barriers before its first and after its last access).
__device__ void plan_of_a_block(Plan& P, const MoeArgs& p) {
  const int n = p.T * p.k, i = threadIdx.x;
  for (int e = i; e < p.E; e += NT) P.first[e] = INT_MAX;
  if (i < FT_PLAN_CAP) P.tokens[i] = 0;
  __syncthreads();
  const int id = i < n ? P.id[i] : -1, slot = slot_of(p, id);
  if (slot >= 0) atomicMin(&P.first[id], i);
  __syncthreads();
  const bool first = slot >= 0 && P.first[id] == i;
  int groups;
  const int rank = block_prefix(first, P.wave_sum, groups);
  if (first) {
    P.first[id] = rank;
    P.slot[rank] = slot;
  }
  __syncthreads();
  const int grp = slot >= 0 ? P.first[id] : -1, token = i / p.k;
  if (i < n) P.grp[i] = grp;
  if (grp >= 0) atomicOr(&P.tokens[grp], 1ull << token);
  __syncthreads();
  const int at = grp >= 0 ? __popcll(P.tokens[grp] & ((1ull << token) - 1)) : 0;
  int pairs;
  const int off = block_prefix(i < groups ? __popcll(P.tokens[i]) : 0, P.wave_sum, pairs);
  if (i <= groups) P.off[i] = off;
  __syncthreads();
  if (grp >= 0) P.pair[P.off[grp] + at] = i;
  if (i == 0) P.groups = groups;
  __syncthreads();
}

// Rows of x and h that are multiplied lie in planes: part v of piece i of a row at place v * pieces + i, so that the 64
// lanes of a load read 64 consecutive 16-byte places.
__device__ __forceinline__ int plane_of(int i, int parts, int pieces) { return i % parts * pieces + i / parts; }
// Element r of a row of fp32 (4 a place).
__device__ __forceinline__ int plane_of_f32(int r, int parts, int pieces) {
  return plane_of(r >> 2, parts, pieces) * 4 + (r & 3);
}
__device__ __forceinline__ void stage_rows(uint4* dst, const uint4* src, int places, int me, int threads) {
  for (int i = me; i < places; i += threads) dst[i] = src[i];
}
template <int NV>
__device__ __forceinline__ void load_parts(uint4 (&v)[NV], const uint4* row, int pieces, int i) {
#pragma unroll
  for (int q = 0; q < NV; ++q) v[q] = row[q * pieces + i];
}

// ---- logits; and by each of the last blocks, where a form multiplies it so, a row of x in planes (MXFP4) or in 8 bits ------
template <int FMT, int TT, int TE>
__global__ __launch_bounds__(256) void moe_logits_kernel(MoeArgs p, const uint16_t* __restrict__ w, float* logits, int eb,
                                                         int blocks) {
  __shared__ uint32_t red[4];
  const int b = blockIdx.x;
  if (b < blocks)
    router_logits_wave<TT, TE>(p.x, w, p.T, p.d, p.E, b / eb * TT, (b % eb * 4 + (threadIdx.x >> 6)) * TE, threadIdx.x & 63, logits);
  else if constexpr (FMT == FT_W_I8)
    quant_row<false, 256, 2>(p.x + (size_t)(b - blocks) * p.d, p.d, static_cast<int8_t*>(p.xv) + (size_t)(b - blocks) * p.d,
                             p.xs + (b - blocks), red);
  else if constexpr (FMT == FT_W_MXFP4) {
    constexpr int NV = Fmt<FMT>::NU;
    const uint4* src = reinterpret_cast<const uint4*>(p.x + (size_t)(b - blocks) * p.d);
    uint4* dst = static_cast<uint4*>(p.xv) + (size_t)(b - blocks) * (p.d / 8);
    for (int i = threadIdx.x; i < p.d / 8; i += 256) dst[plane_of(i, NV, p.d / Fmt<FMT>::E)] = src[i];
  }
}

// Tokens first, first + step, ... one at a time (two of 1024 experts' logits would not fit the registers).
template <int NS>
__device__ __forceinline__ void topk_rows_ns(const MoeArgs& p, int first, int step, int lane, int32_t* id, float* gate) {
  for (int t = first; t < p.T; t += step) {
    TopkIn<NS> in;
    topk_load<NS>(p.logits + (size_t)t * p.E, p.allowed ? p.allowed + (size_t)t * p.E : nullptr, p.E, lane, in);
    topk_pick32<NS>(in, p.k, lane, id + t * p.k, gate + t * p.k);
  }
}
__device__ __forceinline__ void topk_rows(const MoeArgs& p, int first, int step, int lane, int32_t* id, float* gate) {
  if (p.E <= 64)
    topk_rows_ns<1>(p, first, step, lane, id, gate);
  else if (p.E <= 128)
    topk_rows_ns<2>(p, first, step, lane, id, gate);
  else if (p.E <= 256)
    topk_rows_ns<4>(p, first, step, lane, id, gate);
  else
    topk_rows_ns<16>(p, first, step, lane, id, gate);
}
// More than a few tokens: a launch of its own, a wavefront a token (moe_go).
__global__ __launch_bounds__(64) void moe_topk_kernel(MoeArgs p) {
  topk_rows(p, blockIdx.x, gridDim.x, threadIdx.x, p.idx, p.gates);
}

// ---- gate/up ----------------------------------------------------------------------------------
// A wavefront takes units of RG row pairs (gate and up) in turn: every one gets of every group, whose numbers of
// tokens differ.
template <int FMT, int JC, int RG, bool LV>
__device__ __forceinline__ void up_units(const MoeArgs& p, const Plan& P, const uint4* sx) {
  constexpr int E = Fmt<FMT>::E, NV = Fmt<FMT>::NU, TB = 2;
  typedef typename Fmt<FMT>::Acc Acc;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Rec R = rec_of<FMT>(p.d, p.f);
  const int pieces = p.d / E, J = (pieces + 63) >> 6, rb = row_bytes<FMT>(p.d);
  const int per_group = (p.f + RG - 1) / RG;
  const int units = P.groups * per_group;
  for (int u = blockIdx.x * NW + wave; u < units; u += gridDim.x * NW) {
    const int g = u / per_group, r0 = (u - g * per_group) * RG;
    const uint8_t* rp = p.rec + (size_t)__builtin_amdgcn_readfirstlane(P.slot[g]) * p.S;
    const auto rec = buf_rsrc(rp, (uint32_t)p.S);
    const int first = __builtin_amdgcn_readfirstlane(P.off[g]), n = __builtin_amdgcn_readfirstlane(P.off[g + 1]) - first;
    uint4 wg[RG][JC], wu[RG][JC];
    uint32_t sg[RG][JC], su[RG][JC];
    auto load = [&](int j0) {
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const uint32_t row = r0 + r, base = row * (uint32_t)rb, sb = row * (uint32_t)pieces;
#pragma unroll
        for (int j = 0; j < JC; ++j) {
          const int i = (j0 + j) * 64 + lane;
          const bool in = (int)row < p.f && i < pieces;
          wg[r][j] = buf_ld16(rec, in ? base + 16u * i : kOOB);
          wu[r][j] = buf_ld16(rec, in ? R.up + base + 16u * i : kOOB);
          sg[r][j] = FMT == FT_W_MXFP4 ? buf_ld8(rec, in ? R.gs + sb + i : kOOB) : 0;
          su[r][j] = FMT == FT_W_MXFP4 ? buf_ld8(rec, in ? R.us + sb + i : kOOB) : 0;
        }
      }
    };
    load(0);
    for (int tb = 0; tb < n; tb += TB) {
      Acc ag[TB][RG], au[TB][RG];
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int r = 0; r < RG; ++r) ag[t][r] = au[t][r] = 0;
      for (int j0 = 0; j0 < J; j0 += JC) {
        if (J > JC && (j0 > 0 || tb > 0)) load(j0);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          if (tb + t >= n) continue;
          const int tok = __builtin_amdgcn_readfirstlane(P.pair[first + tb + t]) / p.k;
          const uint4* row = (LV ? sx : static_cast<const uint4*>(p.xv)) + (size_t)tok * pieces * NV;
#pragma unroll
          for (int j = 0; j < JC; ++j) {
            const int i = (j0 + j) * 64 + lane;
            if (i >= pieces) continue;
            uint4 v[NV];
            load_parts<NV>(v, row, pieces, i);
#pragma unroll
            for (int r = 0; r < RG; ++r) {
              ag[t][r] = piece_dot<FMT, false, NV>(wg[r][j], sg[r][j], v, ag[t][r]);
              au[t][r] = piece_dot<FMT, false, NV>(wu[r][j], su[r][j], v, au[t][r]);
            }
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        if (tb + t >= n) continue;
        const int pair = __builtin_amdgcn_readfirstlane(P.pair[first + tb + t]);
        wave_totals<RG>(ag[t]);
        wave_totals<RG>(au[t]);
        constexpr int LANES = RG >= 4 ? 16 : RG == 2 ? 32 : 64;  // that hold one total
#pragma unroll
        for (int q = 0; q < (RG + 3) / 4; ++q) {
          const int row = r0 + 4 * q + total_of<RG>(lane);
          if (lane % LANES != 0 || row >= p.f) continue;
          if constexpr (FMT == FT_W_I8) {
            const float *gs = reinterpret_cast<const float*>(rp + R.gs) + row, ts = p.xs[pair / p.k];
            const float v = act_f(i8_value(ag[t][q], gs[0], ts), FT_ACT_SILU) * i8_value(au[t][q], gs[p.f], ts);
            static_cast<uint16_t*>(p.h)[(size_t)pair * p.f + row] = (uint16_t)pack2<false>(v, 0.0f);
          } else {
            static_cast<float*>(p.h)[(size_t)pair * p.f + plane_of_f32(row, Fmt<FMT>::ND, p.f / E)] = silu(ag[t][q]) * au[t][q];
          }
        }
      }
    }
  }
}

// The top-k of all tokens (unless it is there) and their grouping, by every block for itself; the first one leaves both in
// memory.
__device__ __forceinline__ void routes(const MoeArgs& p, Plan& P, int lane, int wave) {
  const int n = p.T * p.k;
  if (!p.ranked) {
    topk_rows(p, wave, NW, lane, P.id, P.gate);
  } else if ((int)threadIdx.x < n) {
    P.id[threadIdx.x] = p.idx[threadIdx.x];
    P.gate[threadIdx.x] = p.gates[threadIdx.x];
  }
  if (p.T > 1) __syncthreads();
  if (n <= 64) {
    if (wave == 0) plan_of_a_wave(P, p, lane);
    __syncthreads();
  } else {
    plan_of_a_block(P, p);
  }
  if (blockIdx.x == 0) {
    const int i = threadIdx.x;
    if (i < n) {
      if (!p.ranked) {
        p.idx[i] = P.id[i];
        p.gates[i] = P.gate[i];
      }
      p.grouped->grp[i] = P.grp[i];
      p.grouped->gate[i] = P.gate[i];
      p.grouped->pair[i] = P.pair[i];  // those past the last are not used
      p.grouped->slot[i] = P.slot[i];
    }
    if (i <= n) p.grouped->off[i] = P.off[i];
    if (i == 0) p.grouped->groups = P.groups;
  }
}

template <int FMT, int JC, int RG>
__global__ __launch_bounds__(NT) void moe_up_kernel(MoeArgs p) {
  __shared__ Plan P;
  extern __shared__ uint4 vec[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (p.lds_vec) {
    // with few tokens, by the wavefronts that have none to rank
    const int skip = p.T <= NW / 2 ? p.T * 64 : 0;
    if ((int)threadIdx.x >= skip)
      stage_rows(vec, static_cast<const uint4*>(p.xv), p.T * (p.d / Fmt<FMT>::E) * Fmt<FMT>::NU, threadIdx.x - skip, NT - skip);
  }
  routes(p, P, lane, wave);
  if (p.lds_vec)
    up_units<FMT, JC, RG, true>(p, P, vec);
  else
    up_units<FMT, JC, RG, false>(p, P, nullptr);
}

// ---- down --------------------------------------------------------------------------------------
// A block owns p.rows rows of every expert's W_down and so of y; its wavefronts take units of RR rows of one
// group.  A pair's results wait in LDS until all are there, then each token's are added in the order of j.
constexpr int kDownRows = 16;

__device__ __forceinline__ void grouped_to_lds(const MoeArgs& p, Grouped& P) {
  const Grouped& G = *p.grouped;
  const int n = p.T * p.k, i = threadIdx.x;
  if (i < n) {
    P.grp[i] = G.grp[i];
    P.gate[i] = G.gate[i];
    P.pair[i] = G.pair[i];
    P.slot[i] = G.slot[i];
  }
  if (i <= n) P.off[i] = G.off[i];
  if (i == 0) P.groups = G.groups;
}
__device__ __forceinline__ void put_y(const MoeArgs& p, size_t at, float s) {
  if (p.y_f32) {
    if (p.res) s += static_cast<const float*>(p.res)[at];
    static_cast<float*>(p.y)[at] = s;
  } else {
    if (p.res) s += to_f32<false>(static_cast<const uint16_t*>(p.res)[at]);
    static_cast<uint16_t*>(p.y)[at] = (uint16_t)pack2<false>(s, 0.0f);
  }
}
// Rows b0 .. b0 + nr of the tokens' sums over the pairs that have a group, from their results: put(token's place, sum).
template <class Put>
__device__ __forceinline__ void sum_experts(const MoeArgs& p, const Grouped& P, const float* out, int b0, int nr, Put put) {
  for (int e = threadIdx.x; e < p.T * nr; e += NT) {
    const int t = e / nr, r = e - t * nr;
    float s = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int q = t * p.k + j;
      if (P.grp[q] >= 0) s = fmaf(P.gate[q], out[q * kDownRows + r], s);
    }
    put((size_t)t * p.d + b0 + r, s);
  }
}

template <int FMT, int JC, int RR, bool LV, class Stage>
__device__ __forceinline__ void down_units(const MoeArgs& p, const Grouped& P, const uint4* sh, const float* hs, float* out,
                                           Stage stage) {
  constexpr int E = Fmt<FMT>::E, NV = Fmt<FMT>::ND, TB = 2;
  typedef typename Fmt<FMT>::Acc Acc;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Rec R = rec_of<FMT>(p.d, p.f);
  const int pieces = p.f / E, J = (pieces + 63) >> 6, rb = row_bytes<FMT>(p.f);
  const int b0 = blockIdx.x * p.rows, nr = min(p.rows, p.d - b0), per_group = (nr + RR - 1) / RR;
  uint4 wv[RR][JC];
  uint32_t sc[RR][JC];
  auto load = [&](const uint8_t* rp, int q0, int j0) {
    const auto rec = buf_rsrc(rp, (uint32_t)p.S);
#pragma unroll
    for (int r = 0; r < RR; ++r) {
      const uint32_t base = R.down + (uint32_t)(b0 + q0 + r) * (uint32_t)rb;
#pragma unroll
      for (int j = 0; j < JC; ++j) {
        const int i = (j0 + j) * 64 + lane;
        const bool in = q0 + r < nr && i < pieces;
        wv[r][j] = buf_ld16(rec, in ? base + 16u * i : kOOB);
        sc[r][j] = FMT == FT_W_MXFP4 ? buf_ld8(rec, in ? R.ds + (uint32_t)(b0 + q0 + r) * (uint32_t)pieces + i : kOOB) : 0;
      }
    }
  };
  const int units = P.groups * per_group;
  bool staged = false;
  // (everyone stages, whether it has a unit or not)
  for (int u = wave; u < units || !staged; u += NW) {
    const bool any = u < units;
    const int g = any ? u / per_group : 0, q0 = (u - g * per_group) * RR;
    const uint8_t* rp = p.rec + (any ? (size_t)__builtin_amdgcn_readfirstlane(P.slot[g]) * p.S : 0);
    if (any) load(rp, q0, 0);
    if (!staged) {
      stage();  // behind the first weights
      staged = true;
    }
    if (!any) break;
    const int first = __builtin_amdgcn_readfirstlane(P.off[g]), n = __builtin_amdgcn_readfirstlane(P.off[g + 1]) - first;
    for (int tb = 0; tb < n; tb += TB) {
      Acc acc[TB][RR];
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int r = 0; r < RR; ++r) acc[t][r] = 0;
      for (int j0 = 0; j0 < J; j0 += JC) {
        if (J > JC && (j0 > 0 || tb > 0)) load(rp, q0, j0);
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          if (tb + t >= n) continue;
          const int pair = __builtin_amdgcn_readfirstlane(P.pair[first + tb + t]);
          const uint4* row = (LV ? sh : static_cast<const uint4*>(FMT == FT_W_I8 ? (const void*)p.hq : p.h)) + (size_t)pair * pieces * NV;
#pragma unroll
          for (int j = 0; j < JC; ++j) {
            const int i = (j0 + j) * 64 + lane;
            if (i >= pieces) continue;
            uint4 v[NV];
            load_parts<NV>(v, row, pieces, i);
#pragma unroll
            for (int r = 0; r < RR; ++r) acc[t][r] = piece_dot<FMT, true, NV>(wv[r][j], sc[r][j], v, acc[t][r]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        if (tb + t >= n) continue;
        const int pair = __builtin_amdgcn_readfirstlane(P.pair[first + tb + t]);
        wave_totals<RR>(acc[t]);
        constexpr int LANES = RR >= 4 ? 16 : RR == 2 ? 32 : 64;
#pragma unroll
        for (int q = 0; q < (RR + 3) / 4; ++q) {
          const int r = q0 + 4 * q + total_of<RR>(lane);
          if (lane % LANES != 0 || r >= nr) continue;
          if constexpr (FMT == FT_W_I8)
            out[pair * kDownRows + r] = i8_value(acc[t][q], reinterpret_cast<const float*>(rp + R.ds)[b0 + r], hs[pair]);
          else
            out[pair * kDownRows + r] = acc[t][q];
        }
      }
    }
  }
}

template <int FMT, int JC, int RR>
__global__ __launch_bounds__(NT) void moe_down_kernel(MoeArgs p) {
  __shared__ Grouped P;
  __shared__ float s_hs[FMT == FT_W_I8 ? FT_PLAN_CAP : 1];
  extern __shared__ uint4 vec[];  // results [pairs][kDownRows], then rows of h
  const int n = p.T * p.k, i = threadIdx.x;
  float* out = reinterpret_cast<float*>(vec);
  uint4* sh = vec + n * kDownRows / 4;
  grouped_to_lds(p, P);
  if (FMT == FT_W_I8 && p.hq && i < n) s_hs[i] = p.hs[i];
  __syncthreads();
  if (p.lds_vec)
    down_units<FMT, JC, RR, true>(p, P, sh, s_hs, out, [&]() {
      if (FMT == FT_W_I8 && !p.hq) {  // few pairs: each block makes the codes of h for itself
        for (int q = threadIdx.x >> 6; q < n; q += NW)
          quant_row<false, 64, 4>(static_cast<const uint16_t*>(p.h) + (size_t)q * p.f, p.f,
                                  reinterpret_cast<int8_t*>(sh) + (size_t)q * p.f, s_hs + q, nullptr);
      } else {
        stage_rows(sh, static_cast<const uint4*>(FMT == FT_W_I8 ? (const void*)p.hq : p.h), n * (p.f / Fmt<FMT>::E) * Fmt<FMT>::ND, i, NT);
      }
      __syncthreads();
    });
  else
    down_units<FMT, JC, RR, false>(p, P, nullptr, s_hs, out, []() {});
  __syncthreads();
  const int b0 = blockIdx.x * p.rows;
  sum_experts(p, P, out, b0, min(p.rows, p.d - b0), [&](size_t at, float s) { put_y(p, at, s); });
}

// ---- many tokens an expert: matrix instructions ----------------------------------------------------
// The same products for groups of several tokens, cut into parts of up to 16: a tile is 16 rows of an expert (gate/up: 8
// of each) and the tokens of a part, weights as the MFMA's second operand, so that each is loaded and converted
// once a part.  Lane l: row (and token) l % 16, in a step the k of its quarter l / 16.  KW wavefronts share a tile's
// chunks and add their sums in LDS; the block's others take further tiles.  The next chunk, of this tile or the next one,
// is on its way while one is multiplied, each load leaving as its registers are used up.
//   bf16   v_mfma_f32_16x16x32_bf16
//   MXFP4  the same on codes turned into bf16 exactly; a step is one block of 32, whose scale multiplies its
//          fp32 sum; exchanges across the wave bring a lane's block to the quarters
//   8-bit  v_mfma_i32_16x16x64_i8
// h stays fp32 for bf16 and MXFP4: it is cut into three bf16 numbers whose sum it is (8 + 8 + 8 bits), each with its own
// MFMA; the matrix cores have room for that.
// Loads of 64 bytes from each of 16 rows, as the weights', cost the load unit four times what 1 KB in a line does, so the
// tokens' operands do not come that way: gate/up holds a part's x in LDS, and h lies in memory as down multiplies it (frag_place).
// 64 tokens, 32 an expert, d = 2048, d_ff = 768 in bf16: with both gathered 185 us, so 107 (gate/up 48, 100 MB of weights read
// once per 16 tokens; down 43, each block reading all of h).
template <int FMT>
struct Many {
  static constexpr int KS = FMT == FT_W_I8 ? 64 : 32;   // k of a step
  static constexpr int EB = FMT == FT_W_I8 ? 1 : 2;     // bytes of an element of x
  static constexpr int PARTS = FMT == FT_W_I8 ? 1 : 3;  // of h
  static constexpr int HL = FMT == FT_W_I8 ? 1 : 2;     // 16 bytes of h a lane multiplies in a step
  typedef typename std::conditional<FMT == FT_W_I8, int, float>::type One;
  typedef typename std::conditional<FMT == FT_W_I8, i32x4_t, f32x4_t>::type Acc;
};
// Where a lane's weights of a chunk are: a row of n elements at byte `base` of a record (scales at sbase), chunk `chunk` of it.
struct ManyAt {
  __amdgpu_buffer_rsrc_t rec;
  uint32_t base, sbase;
  int n, chunk, g;
  bool in;
};
// A lane's weights of a chunk of ST steps; zeros past a row's end.
template <int FMT, int ST>
struct ManyWeights {
  static constexpr int KS = Many<FMT>::KS, PER = FMT == FT_W_MXFP4 ? 4 : 1, WL = ST / PER;  // steps a load has, loads
  uint4 w[WL];
  uint32_t sc[FMT == FT_W_MXFP4 ? WL : 1];
  __device__ __forceinline__ void load(const ManyAt& a, int l) {
    if constexpr (FMT == FT_W_MXFP4) {
      const int k = (a.chunk * WL + l) * 128;  // n is a multiple of 128
      const bool in = a.in && k < a.n;
      w[l] = buf_ld16(a.rec, in ? a.base + (uint32_t)((k + a.g * 32) >> 1) : kOOB);
      sc[l] = __builtin_amdgcn_raw_buffer_load_b32(a.rec, (int)(in ? a.sbase + (uint32_t)(k >> 5) : kOOB), 0, 0);
    } else {
      const int k = (a.chunk * ST + l) * KS + a.g * (KS / 4);
      w[l] = buf_ld16(a.rec, a.in && k < a.n ? a.base + (uint32_t)(k * Many<FMT>::EB) : kOOB);
    }
  }
  // Each load's steps, and in its place that of `next`: the chunk's loads stay on their way all the time.  x(j, q): part q of
  // the tokens' operand of step j; used(j): x(j, .) is not asked for any more.
  template <int PARTS, class X, class Used>
  __device__ __forceinline__ void multiply(typename Many<FMT>::Acc& acc, const ManyAt& next, X x, Used used) {
#pragma unroll
    for (int l = 0; l < WL; ++l) {
      if constexpr (FMT != FT_W_MXFP4) {
        const i32x4_t wl = __builtin_bit_cast(i32x4_t, w[l]);
#pragma unroll
        for (int q = PARTS - 1; q >= 0; --q) {
          if constexpr (FMT == FT_W_I8)
            acc = mfma16(x(l, q), wl, acc);
          else
            acc = mfma16<false>(x(l, q), wl, acc);
        }
        load(next, l);
        used(l);
      } else {
        // word j of quarter g to quarter j, word g
        uint32_t v[4] = {w[l].x, w[l].y, w[l].z, w[l].w};
        const uint32_t s4 = sc[l];
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
        s32(v[0], v[2]);
        s32(v[1], v[3]);
        s16(v[0], v[1]);
        s16(v[2], v[3]);
        load(next, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const i32x4_t wj = {__builtin_bit_cast(int, mx_pair<0>(v[j])), __builtin_bit_cast(int, mx_pair<1>(v[j])),
                              __builtin_bit_cast(int, mx_pair<2>(v[j])), __builtin_bit_cast(int, mx_pair<3>(v[j]))};
          f32x4_t s = {};
#pragma unroll
          for (int q = PARTS - 1; q >= 0; --q) s = mfma16<false>(x(4 * l + j, q), wj, s);
          const float scale = e8m0((s4 >> (8 * j)) & 255u);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(scale, s[i], acc[i]);
          used(4 * l + j);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The groups in parts.
struct Parts {
  int32_t n;
  int32_t slot[FT_PLAN_CAP];
  uint16_t pair[FT_PLAN_CAP];                  // by group
  uint16_t first[FT_PLAN_CAP], off[FT_PLAN_CAP];  // a part's first place among them, its group's
  uint8_t pairs[FT_PLAN_CAP], of[FT_PLAN_CAP];    // its pairs, its group's (64 tokens at most)
  int32_t wave_sum[NW];
};
// Parts of up to `most` pairs of the groups that take(i) holds for.  All threads of the block, a barrier behind the groups' last
// change; barriers within and behind.
template <class Take>
__device__ void cut_groups(Parts& Q, const Grouped& P, int most, Take take) {
  const int i = threadIdx.x, n = i < P.groups && take(i) ? P.off[i + 1] - P.off[i] : 0;
  int total;
  const int at = block_prefix((n + most - 1) / most, Q.wave_sum, total);
  for (int t = 0; t * most < n; ++t) {
    Q.slot[at + t] = P.slot[i];
    Q.first[at + t] = (uint16_t)(P.off[i] + t * most);
    Q.pairs[at + t] = (uint8_t)min(most, n - t * most);
    Q.off[at + t] = (uint16_t)P.off[i];
    Q.of[at + t] = (uint8_t)n;
  }
  if (i < P.off[P.groups]) Q.pair[i] = (uint16_t)P.pair[i];
  if (i == 0) Q.n = total;
  __syncthreads();
}

// Where h of a group's token i lies (of n, the first of them `off` among the pairs by group), for down: the group's 16 tokens
// of a part side by side, 16 bytes of each in turn.  Byte `at` of its row of `row` bytes:
__device__ __forceinline__ size_t frag_place(int off, int n, int i, size_t row, uint32_t at) {
  const int part = i & ~15, w = min(16, n - part);
  return (size_t)(off + part) * row + ((size_t)(at >> 4) * w + (i & 15)) * 16 + (at & 15);
}

// The wavefronts that share a tile of n elements a row: two chunks each, where there are as many.
template <int FMT, int ST>
__device__ __forceinline__ int kw_log_of(int n) {
  constexpr int CK = ST * Many<FMT>::KS;
  const int chunks = (n + CK - 1) / CK;
  return chunks >= 32 ? 4 : chunks >= 16 ? 3 : chunks >= 8 ? 2 : chunks >= 4 ? 1 : 0;
}

constexpr int kManyPad = 16;  // bytes between rows of x in LDS: 16 tokens' pieces start on different banks

// p.rows: tokens of a part, as many as LDS holds x of.  A block takes consecutive tiles, `per` of one part at a time: it loads
// x once or twice.
template <int FMT>
__global__ __launch_bounds__(NT) void moe_up_many_kernel(MoeArgs p) {
  constexpr int EB = Many<FMT>::EB, KS = Many<FMT>::KS, ST = 8, CK = ST * KS;
  typedef typename Many<FMT>::One One;
  __shared__ Parts Q;
  __shared__ One red[NW * 256];
  extern __shared__ uint4 vec[];  // the plan, then a part's rows of x
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n16 = lane & 15, g = lane >> 4;
  const uint8_t* x = static_cast<const uint8_t*>(FMT == FT_W_I8 ? p.xv : (const void*)p.x);
  {
    Plan& P = *reinterpret_cast<Plan*>(vec);
    routes(p, P, lane, wave);
    cut_groups(Q, P, p.rows, [](int) { return true; });
  }
  const Rec R = rec_of<FMT>(p.d, p.f);
  const int per_part = p.f / 8, rb = row_bytes<FMT>(p.d);  // f % 8 == 0
  const int kw_log = kw_log_of<FMT, ST>(p.d), KW = 1 << kw_log, kw = wave & (KW - 1), per = NW >> kw_log, mine = wave >> kw_log;
  const int chunks = (p.d + CK - 1) / CK, batches = (per_part + per - 1) / per, units = Q.n * batches;  // KW chunks or more
  const int pieces = p.d * EB / 16, xrow = p.d * EB + kManyPad;
  const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
  ManyWeights<FMT, ST> w;
  auto place = [&](int u, int c, bool any) {
    const int q = u / batches, i = (u - q * batches) * per + mine, row = min(i, per_part - 1) * 8 + (n16 & 7);
    const uint8_t* rp = p.rec + (size_t)__builtin_amdgcn_readfirstlane(Q.slot[q]) * p.S;
    return ManyAt{buf_rsrc(rp, (uint32_t)p.S), (n16 < 8 ? 0u : R.up) + (uint32_t)row * (uint32_t)rb,
                  (n16 < 8 ? R.gs : R.us) + (uint32_t)row * (uint32_t)(p.d / 32), p.d, c, g, any && i < per_part};
  };
  if (u0 < u1) {
    const ManyAt at = place(u0, kw, true);
#pragma unroll
    for (int l = 0; l < ManyWeights<FMT, ST>::WL; ++l) w.load(at, l);
  }
  int staged = -1;
  for (int u = u0; u < u1; ++u) {
    const int q = u / batches, n = __builtin_amdgcn_readfirstlane((int)Q.pairs[q]), first = __builtin_amdgcn_readfirstlane((int)Q.first[q]);
    if (q != staged) {  // (nobody reads the rows of the part before: a barrier ended its last unit)
      staged = q;
      const int segs = (pieces + 63) >> 6, all = n * segs;
      for (int s0 = wave; s0 < all; s0 += 4 * NW) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = min(s0 + e * NW, all - 1), r = s / segs, i = min((s - r * segs) * 64 + lane, pieces - 1);
          v[e] = reinterpret_cast<const uint4*>(x + (size_t)(Q.pair[first + r] / p.k) * p.d * EB)[i];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = s0 + e * NW, r = s / segs, i = (s - r * segs) * 64 + lane;
          if (s < all && i < pieces) vec[r * (xrow / 16) + i] = v[e];
        }
      }
      __syncthreads();
    }
    const uint8_t* xr = reinterpret_cast<const uint8_t*>(vec) + min(n16, n - 1) * xrow;
    typename Many<FMT>::Acc acc = {};
    for (int c = kw; c < chunks; c += KW) {
      const bool here = c + KW < chunks, more = here || u + 1 < u1;
      const ManyAt next = place(here || !more ? u : u + 1, here ? c + KW : kw, more);
      w.template multiply<1>(acc, next, [&](int j, int) {
        const int k = (c * ST + j) * KS + g * (16 / EB);
        i32x4_t v = *reinterpret_cast<const i32x4_t*>(xr + (k < p.d ? k * EB : 0));
        if (k >= p.d) v = i32x4_t{};  // x may be an infinity there
        return v;
      }, [](int) {});
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave * 256 + (4 * g + i) * 16 + n16] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < per * 128; e += NT) {
      const int i = (u - q * batches) * per + (e >> 7), tk = (e >> 3) & 15, r = e & 7;
      if (i >= per_part || tk >= n) continue;
      const One* s = red + (e >> 7) * KW * 256 + tk * 16 + r;
      One a = 0, b = 0;
      for (int w = 0; w < KW; ++w) {
        a += s[w * 256];
        b += s[w * 256 + 8];
      }
      const int pair = Q.pair[first + tk], row = i * 8 + r;
      if constexpr (FMT == FT_W_I8) {
        const float* gs = reinterpret_cast<const float*>(p.rec + (size_t)Q.slot[q] * p.S + R.gs) + row;
        const float ts = p.xs[pair / p.k], v = act_f(i8_value(a, gs[0], ts), FT_ACT_SILU) * i8_value(b, gs[p.f], ts);
        static_cast<uint16_t*>(p.h)[(size_t)pair * p.f + row] = (uint16_t)pack2<false>(v, 0.0f);
      } else {
        const int off = Q.off[q];
        float* h = static_cast<float*>(p.h);
        h[frag_place(off, Q.of[q], first - off + tk, (size_t)p.f * 4, (uint32_t)row * 4) >> 2] = silu(a) * b;
      }
    }
    __syncthreads();
  }
}

// 8-bit records: h's codes, a row by each block, where down multiplies them.
__global__ __launch_bounds__(256) void moe_codes_kernel(MoeArgs p) {
  __shared__ uint32_t red[4];
  const Grouped& G = *p.grouped;
  const int at = blockIdx.x;
  if (at >= G.off[G.groups]) return;  // the whole block
  const int pair = G.pair[at], grp = G.grp[pair], off = G.off[grp], n = G.off[grp + 1] - off;
  quant_row<false, 256, 2>(static_cast<const uint16_t*>(p.h) + (size_t)pair * p.f, p.f,
                           [&](int i) { return reinterpret_cast<uint2*>(p.hq + frag_place(off, n, at - off, p.f, (uint32_t)i * 8)); },
                           p.hs + pair, red);
}

// Eight numbers of fp32 as three bf16 each, from the top: the upper 8 bits of what is left.
__device__ __forceinline__ void cut3(const i32x4_t (&v)[2], i32x4_t (&x)[3]) {
  float r[8], m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r[e] = __int_as_float(v[e >> 2][e & 3]);
    m = fmaxf(m, fabsf(r[e]));
  }
  const bool inf = m == INFINITY;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[q][e] = (int)__builtin_amdgcn_perm(__float_as_uint(r[2 * e + 1]), __float_as_uint(r[2 * e]), 0x07060302u);
    if (q == 2) break;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float top = __uint_as_float(__float_as_uint(r[e]) & 0xffff0000u);
      r[e] -= top;
      if (q == 0 && inf && fabsf(top) == INFINITY) r[e] = 0.0f;
    }
  }
}

// A block owns 16 rows of y and, of p.split blocks that share them, the experts e with e % p.split its own number; what each of
// several has of y's sums goes to p.part [split, T, d] (moe_join_kernel).  By the expert's number, so that the order of a token's
// sum hangs on its own experts alone: parts dealt out evenly add it up by what the other tokens take.  It costs next to nothing (64
// tokens, us dealt evenly / by expert: d = 2048, d_ff = 768, 16 experts, k = 8, bf16 106.8 / 107.2; d = 1024, d_ff = 512, 64 experts, k = 6,
// 68.1 / 68.2) but where each of fewer experts than blocks is taken by every token (d = 256, d_ff = 2048, 8 of 8 experts 47.3 / 50.5).
template <int FMT>
__global__ __launch_bounds__(NT) void moe_down_many_kernel(MoeArgs p) {
  constexpr int EB = FMT == FT_W_I8 ? 1 : 4;  // bytes of an element of h
  constexpr int KS = Many<FMT>::KS, PARTS = Many<FMT>::PARTS, HL = Many<FMT>::HL, ST = FMT == FT_W_I8 ? 8 : 4, CK = ST * KS;
  typedef typename Many<FMT>::One One;
  __shared__ Grouped P;
  __shared__ Parts Q;
  __shared__ One red[2][NW * 256];
  extern __shared__ uint4 vec[];  // results [pairs][kDownRows]
  float* out = reinterpret_cast<float*>(vec);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n16 = lane & 15, g = lane >> 4;
  const Rec R = rec_of<FMT>(p.d, p.f);
  const int rb = row_bytes<FMT>(p.f), share = blockIdx.x % p.split, b0 = blockIdx.x / p.split * 16, nr = min(16, p.d - b0);
  grouped_to_lds(p, P);
  // the others' pairs have no group here (each thread's own entry)
  if ((int)threadIdx.x < p.T * p.k && p.split > 1 && p.idx[threadIdx.x] % p.split != share) P.grp[threadIdx.x] = -1;
  __syncthreads();
  cut_groups(Q, P, 16, [&](int i) { return P.grp[P.pair[P.off[i]]] >= 0; });
  const int tiles = Q.n;
  const uint8_t* h = static_cast<const uint8_t*>(FMT == FT_W_I8 ? (const void*)p.hq : p.h);
  const int kw_log = kw_log_of<FMT, ST>(p.f), KW = 1 << kw_log, kw = wave & (KW - 1), per = NW >> kw_log, mine = wave >> kw_log;
  const int chunks = (p.f + CK - 1) / CK;  // KW or more
  ManyWeights<FMT, ST> w;
  i32x4_t x[ST][HL];
  struct Place {
    ManyAt w;
    const uint8_t* row;
    int step;  // bytes from piece to piece
  };
  auto place = [&](int i, int c) {
    const bool any = i < tiles;
    const int q = any ? i : 0, n = Q.pairs[q];
    const uint8_t* rp = p.rec + (size_t)__builtin_amdgcn_readfirstlane(Q.slot[q]) * p.S;
    return Place{ManyAt{buf_rsrc(rp, (uint32_t)p.S), R.down + (uint32_t)(b0 + n16) * (uint32_t)rb,
                        R.ds + (uint32_t)(b0 + n16) * (uint32_t)(p.f / 32), p.f, c, g, any && n16 < nr},
                 // a part as frag_place has it: piece by piece, of each its n tokens
                 h + (size_t)Q.first[q] * p.f * EB + min(n16, n - 1) * 16, n * 16};
  };
  auto load_x = [&](const Place& a, int j) {
    const int k = (a.w.chunk * ST + j) * KS + g * (KS / 4);
#pragma unroll
    for (int e = 0; e < HL; ++e) x[j][e] = *reinterpret_cast<const i32x4_t*>(a.row + ((k < p.f ? k * EB >> 4 : 0) + e) * a.step);
  };
  if (tiles > 0) {
    const Place at = place(mine, kw);
#pragma unroll
    for (int l = 0; l < ManyWeights<FMT, ST>::WL; ++l) w.load(at.w, l);
#pragma unroll
    for (int j = 0; j < ST; ++j) load_x(at, j);
  }
  int buf = 0;
  for (int b = 0; b < tiles; b += per) {
    typename Many<FMT>::Acc acc = {};
    for (int c = kw; c < chunks; c += KW) {
      const bool here = c + KW < chunks;
      const Place next = place(here ? b + mine : b + per < tiles ? b + per + mine : tiles, here ? c + KW : kw);
      i32x4_t x3[3];
      w.template multiply<PARTS>(
          acc, next.w,
          [&](int j, int e) {
            if constexpr (FMT == FT_W_I8) {
              return x[j][0];
            } else {
              if (e == PARTS - 1) {  // asked for first
                if ((c * ST + j) * KS + g * (KS / 4) >= p.f) x[j][0] = x[j][1] = i32x4_t{};  // h may be an infinity there
                cut3(x[j], x3);
              }
              return x3[e];
            }
          },
          [&](int j) { load_x(next, j); });
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[buf][wave * 256 + (4 * g + i) * 16 + n16] = acc[i];
    __syncthreads();  // (the other buffer's sums were read before everyone came here)
    for (int e = threadIdx.x; e < per * 256; e += NT) {
      const int q = b + (e >> 8), tk = (e >> 4) & 15, r = e & 15;
      if (q >= tiles || tk >= Q.pairs[q] || r >= nr) continue;
      const One* s = red[buf] + (e >> 8) * KW * 256 + tk * 16 + r;
      One a = 0;
      for (int w = 0; w < KW; ++w) a += s[w * 256];
      const int pair = Q.pair[Q.first[q] + tk];
      if constexpr (FMT == FT_W_I8)
        out[pair * kDownRows + r] =
            i8_value(a, reinterpret_cast<const float*>(p.rec + (size_t)Q.slot[q] * p.S + R.ds)[b0 + r], p.hs[pair]);
      else
        out[pair * kDownRows + r] = a;
    }
    buf ^= 1;
  }
  __syncthreads();
  sum_experts(p, P, out, b0, nr, [&](size_t at, float s) {
    if (p.split > 1)
      p.part[(size_t)share * p.T * p.d + at] = s;
    else
      put_y(p, at, s);
  });
}

__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs p) {
  const int n = p.T * p.d, at = blockIdx.x * 256 + threadIdx.x;
  if (at >= n) return;
  float s = 0.0f;
  for (int i = 0; i < p.split; ++i) s += p.part[(size_t)i * n + at];
  put_y(p, at, s);
}

// ---- launches -----------------------------------------------------------------------------------
constexpr int kUnits = 256;           // compute units
constexpr size_t kVecLds = 136 << 10;  // most of a block's LDS for rows of x, or for results and rows of h
// gate/up's matrix form: a part's x, beside the parts and sums (16 tokens of d = 4096 in bf16 take 128 KB)
constexpr size_t kManyLds = 136 << 10;
static_assert(sizeof(Plan) <= kManyLds && kManyLds + sizeof(Parts) + NW * 1024 <= 160 << 10, "");
// Elements of a row of h, and of all of h, up to which each block of the down product makes h's codes itself, in place of a launch
// for all.  A row goes to one wavefront, which holds 2048 elements and reads the rest twice (us of a layer, itself against the
// launch, d = 4096, one token, 1 / 2 / 4 rows: of 2048 19.2 / 20.7, 24.8 / 26.8, 32.3 / 35.6; of 4096 24.6 / 24.6, 35.4 / 36.0,
// 52.9 / 54.1; of 6144 30.4 / 28.4, 46.4 / 45.5, 72.1 / 72.3; one of 8192 35.6 / 32.4, of 14336 51.6 / 42.7, of 24576 85.3 / 67.2;
// rows of 768 and 2048: 6144 elements 20.9 / 22.6, 12288 37.4 / 40.5, 24576 46.1 / 46.2 and 61.6 / 65.6, 36864 58.9 / 57.2,
// 79872 88.7 / 83.1).
constexpr int kOwnRow = 4096;
constexpr size_t kOwnRows = 24 << 10;

// Whether the experts that are taken are taken by enough tokens for the matrix forms: as many as T tokens with k of E each
// meet if all are equally likely, allowed and given a record (by the shape and T alone, as the order of sums is; where a few experts take
// most tokens, the rows' form runs past the point where the other is faster).  How many are enough goes by the rows' length (d + d_ff), which fills the rows' form's loads
// and not the other's, and by the elements that the layer reads, against the matrix form's longer way to its first
// product (MXFP4, whose conversions it saves, gains all the same).  us of rows against matrix form at so many tokens an expert:
//                        bf16                         MXFP4                                8-bit
//   1024 x 512 of 16..128  2.3 43 / 46, 4 52 / 47     2.2 38 / 34, 3.2 171 / 74              2.3 56 / 51, 4 53 / 44
//   2048 x 768 of 128    2.7 240 / 251, 4.1 291 / 260   2.3 146 / 147, 2.7 178 / 158, 4.1 255 / 162   2.7 140 / 141, 4.1 170 / 145
//   2048 x 768 of 8      4 43 / 47, 8 61 / 51         4 48 / 38                            4 36 / 41, 8 49 / 42
//   4096 x 2048 of 64    3.1 714 / 634, 6 1030 / 669   3.1 326 / 369, 3.8 378 / 371         3.1 315 / 307, 6 430 / 307
//   256 x 128 of 64      8 82 / 38                    8 - / 35                             8 79 / 41
//   4096 x 14336 of 8    4 752 / 546                  3.1 265 / 321, 4 336 / 323             3.1 302 / 275, 4 368 / 277
template <int FMT>
bool many_tokens(const MoeArgs& A) {
  const double pairs = (double)A.T * A.k, met = A.E * (1.0 - pow(1.0 - (double)A.k / A.E, A.T)), row = A.d + A.f;
  const double read = met * A.d * A.f, start = std::min(1.5, 16.7e6 / read);
  const double least = FMT == FT_W_BF16    ? 2.8 + start
                       : FMT == FT_W_MXFP4 ? std::min(3.9, 1.55 + row / 2700)
                                           : std::min(2.7, 0.1 + row / 1000) + start;
  return pairs > least * met;
}

// A lane holds W pieces of weights at once: rows of up to 64 JC pieces in one go, the longer the fewer of them.
template <int FMT, int W>
int moe_go(MoeArgs A, bool many, hipStream_t s) {
  const size_t P = (size_t)A.T * A.k;
  const size_t xb = (size_t)A.T * A.d * (FMT == FT_W_I8 ? 1 : 2);
  constexpr int E = Fmt<FMT>::E;
  A.rows = (A.d + kUnits - 1) / kUnits;
  if (A.rows > kDownRows) A.rows = kDownRows;
  const unsigned down_blocks = (unsigned)((A.d + A.rows - 1) / A.rows);
  if (many) {
    const size_t row = (size_t)A.d * (FMT == FT_W_I8 ? 1 : 2) + kManyPad;
    const size_t fit = kManyLds / row, part = fit < 16 ? fit : 16;  // 4 or more: d <= 16384
    const size_t lds = (part < (size_t)A.T ? part : A.T) * row;
    MoeArgs up = A;
    up.rows = (int)part;
    hipLaunchKernelGGL(moe_up_many_kernel<FMT>, dim3(kUnits), dim3(NT), lds > sizeof(Plan) ? lds : sizeof(Plan), s, up);
    if (int st = launched("moe_up_many_kernel")) return st;
    if (FMT == FT_W_I8) {
      hipLaunchKernelGGL(moe_codes_kernel, dim3((unsigned)P), dim3(256), 0, s, A);
      if (int st = launched("moe_codes_kernel")) return st;
    }
    A.split = moe_down_split(A.d, A.E);
    hipLaunchKernelGGL(moe_down_many_kernel<FMT>, dim3((unsigned)((A.d + 15) / 16 * A.split)), dim3(NT), P * kDownRows * 4, s, A);
    if (A.split == 1) return launched("moe_down_many_kernel");
    if (int st = launched("moe_down_many_kernel")) return st;
    hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((A.T * A.d + 255) / 256)), dim3(256), 0, s, A);
    return launched("moe_join_kernel");
  }
  A.lds_vec = xb <= kVecLds;
  auto up = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(kUnits), dim3(NT), A.lds_vec ? xb : 0, s, A); };
  const int ju = (A.d / E + 63) / 64;
  if constexpr (FMT == FT_W_MXFP4) {
    ju > 1 ? up(moe_up_kernel<FMT, 2, W / 4>) : up(moe_up_kernel<FMT, 1, W / 2>);
  } else {
    if (FMT == FT_W_BF16 && ju > 4)
      up(moe_up_kernel<FT_W_BF16, 8, 1>);
    else
      ju > 2 ? up(moe_up_kernel<FMT, 4, W / 8>) : ju > 1 ? up(moe_up_kernel<FMT, 2, W / 4>) : up(moe_up_kernel<FMT, 1, W / 2>);
  }
  if (int st = launched("moe_up_kernel")) return st;
  const size_t hb = P * A.f * (FMT == FT_W_I8 ? 1 : 4), ob = P * kDownRows * 4;
  A.lds_vec = hb <= kVecLds - ob;
  if (FMT == FT_W_I8) {
    if (A.f <= kOwnRow && P * A.f <= kOwnRows && A.lds_vec)
      A.hq = nullptr;
    else if (int st = launch_i8_quant(static_cast<const uint16_t*>(A.h), A.f, (int)P, A.f, false, A.hq, A.hs, s))
      return st;
  }
  auto down = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(down_blocks), dim3(NT), ob + (A.lds_vec ? hb : 0), s, A);
  };
  const int jd = (A.f / E + 63) / 64;
  if constexpr (FMT == FT_W_MXFP4)
    jd > 1 ? down(moe_down_kernel<FMT, 2, W / 2>) : down(moe_down_kernel<FMT, 1, W>);
  else
    jd > 2 ? down(moe_down_kernel<FMT, 4, W / 4>) : jd > 1 ? down(moe_down_kernel<FMT, 2, W / 2>) : down(moe_down_kernel<FMT, 1, 8>);
  return launched("moe_down_kernel");
}

}  // namespace

int launch_moe_layer(const MoeLayer& L, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (L.T <= 0) return FT_OK;
  MoeArgs A{};
  A.x = L.x;
  A.logits = L.logits;
  A.allowed = L.allowed;
  A.rec = L.records;
  A.slot_of = L.slot_of;
  A.T = L.T;
  A.d = L.d;
  A.f = L.d_ff;
  A.E = L.E;
  A.k = L.k;
  A.n_slots = L.n_slots;
  A.S = L.S;
  A.idx = L.idx;
  A.gates = L.gates;
  A.grouped = static_cast<Grouped*>(L.grouped);
  A.xv = L.fmt == FT_W_BF16 ? const_cast<uint16_t*>(L.x) : L.xv;
  A.xs = L.xs;
  A.hq = L.hq;
  A.hs = L.hs;
  A.h = L.h;
  A.part = L.part;
  A.res = L.res;
  A.y = L.y;
  A.y_f32 = L.y_f32;
  // every block ranks all tokens for itself up to 24 (us of a layer, itself against a launch more: 16 tokens 62.0 / 62.7, 32
  // 85.3 / 83.6, 64 142 / 135, of few experts 66.8 / 62.9)
  A.ranked = A.T > 24;
  // few logits a wavefront: their sums run in a fixed order and so one behind the other
  const int tt = L.T == 1 ? 1 : L.T <= 16 ? 2 : 4, te = L.T == 1 ? 1 : 2;
  const int eb = (L.E + 4 * te - 1) / (4 * te), blocks = eb * ((L.T + tt - 1) / tt);
  const bool many = L.fmt == FT_W_BF16 ? many_tokens<FT_W_BF16>(A) : L.fmt == FT_W_MXFP4 ? many_tokens<FT_W_MXFP4>(A) : many_tokens<FT_W_I8>(A);
  const bool rows = L.fmt == FT_W_I8 || (L.fmt == FT_W_MXFP4 && !many);  // the matrix form reads 16-bit x as it is
  const dim3 grid((unsigned)(blocks + (rows ? L.T : 0)));
  auto logits = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, A, L.w_router, L.logits, eb, blocks); };
  auto by_format = [&](auto bf16, auto mx, auto i8) { L.fmt == FT_W_BF16 ? logits(bf16) : L.fmt == FT_W_MXFP4 ? logits(mx) : logits(i8); };
  if (tt == 1)
    by_format(moe_logits_kernel<FT_W_BF16, 1, 1>, moe_logits_kernel<FT_W_MXFP4, 1, 1>, moe_logits_kernel<FT_W_I8, 1, 1>);
  else if (tt == 2)
    by_format(moe_logits_kernel<FT_W_BF16, 2, 2>, moe_logits_kernel<FT_W_MXFP4, 2, 2>, moe_logits_kernel<FT_W_I8, 2, 2>);
  else
    by_format(moe_logits_kernel<FT_W_BF16, 4, 2>, moe_logits_kernel<FT_W_MXFP4, 4, 2>, moe_logits_kernel<FT_W_I8, 4, 2>);
  if (int st = launched("moe_logits_kernel")) return st;
  if (A.ranked) {
    hipLaunchKernelGGL(moe_topk_kernel, dim3((unsigned)A.T), dim3(64), 0, s, A);
    if (int st = launched("moe_topk_kernel")) return st;
  }
  if (L.fmt == FT_W_I8) return moe_go<FT_W_I8, 16>(A, many, s);
  if (L.fmt == FT_W_MXFP4) return moe_go<FT_W_MXFP4, 8>(A, many, s);
  return moe_go<FT_W_BF16, 16>(A, many, s);
}

}  // namespace ft

// Device parts of the router that several kernels share (kernels.hip, kernels_moe.hip): a wavefront's
// logits in their fixed order, and the top-k with its gates.  gfx950 only.
#pragma once

#include "device_common.h"

namespace ft {
namespace dev {

__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ uint4 keep_if(uint4 v, bool c) {
  return make_uint4(c ? v.x : 0u, c ? v.y : 0u, c ? v.z : 0u, c ? v.w : 0u);
}

// Logits by one wavefront: the TE experts from e0 on for the TT tokens from t0 on, in the order that
// router_logits_kernel states (lane l owns elements (i mod 512) / 8 == l, adds its products in
// increasing i, then a butterfly), loading JB chunks of 512 elements per operand at once.
template <int TT, int TE>
__device__ __forceinline__ void router_logits_wave(const uint16_t* __restrict__ x, const uint16_t* __restrict__ w, int T,
                                                   int d, int E, int t0, int e0, int lane, float* __restrict__ logits) {
  constexpr int JB = 40 / (TT + TE) < 8 ? 40 / (TT + TE) : 8;  // at most 40 16-byte loads in flight
  if (e0 >= E) return;
  float acc[TT][TE];
#pragma unroll
  for (int a = 0; a < TT; ++a)
#pragma unroll
    for (int b = 0; b < TE; ++b) acc[a][b] = 0.0f;
  const int J = (d + 511) >> 9;
  for (int j0 = 0; j0 < J; j0 += JB) {
    // every load is issued unconditionally from a clamped (in-bounds) address and
    // the operands past the ends are zeroed afterwards: loads under a branch come
    // out one behind the other
    uint4 xv[JB][TT], wv[JB][TE];
#pragma unroll
    for (int jj = 0; jj < JB; ++jj) {
      const int i0 = (j0 + jj) * 512 + lane * 8;
      const bool in = j0 + jj < J && i0 < d;
      const int ic = in ? i0 : 0;
#pragma unroll
      for (int a = 0; a < TT; ++a) {
        const int ta = t0 + a < T ? t0 + a : T - 1;
        xv[jj][a] = ld16(x + (size_t)ta * d + ic);
      }
#pragma unroll
      for (int b = 0; b < TE; ++b) {
        const int eb = e0 + b < E ? e0 + b : E - 1;
        wv[jj][b] = ld16(w + (size_t)eb * d + ic);
      }
    }
    // only the positions past d need zeros (as in router_logits_kernel); the
    // logits of tokens and experts past the ends are not stored
#pragma unroll
    for (int jj = 0; jj < JB; ++jj) {
      const bool in = j0 + jj < J && (j0 + jj) * 512 + lane * 8 < d;
#pragma unroll
      for (int a = 0; a < TT; ++a) xv[jj][a] = keep_if(xv[jj][a], in);
#pragma unroll
      for (int b = 0; b < TE; ++b) wv[jj][b] = keep_if(wv[jj][b], in);
    }
#pragma unroll
    for (int jj = 0; jj < JB; ++jj) {
      if (j0 + jj >= J) continue;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
#pragma unroll
        for (int a = 0; a < TT; ++a) {
          const uint32_t xw = (r >> 1) == 0 ? xv[jj][a].x : (r >> 1) == 1 ? xv[jj][a].y
                            : (r >> 1) == 2 ? xv[jj][a].z : xv[jj][a].w;
          const float xf = (r & 1) ? bf_hi(xw) : bf_lo(xw);
#pragma unroll
          for (int b = 0; b < TE; ++b) {
            const uint32_t ww = (r >> 1) == 0 ? wv[jj][b].x : (r >> 1) == 1 ? wv[jj][b].y
                              : (r >> 1) == 2 ? wv[jj][b].z : wv[jj][b].w;
            const float wf = (r & 1) ? bf_hi(ww) : bf_lo(ww);
            acc[a][b] = acc[a][b] + xf * wf;  // same order as router_logits_kernel
          }
        }
      }
    }
  }
#pragma unroll
  for (int a = 0; a < TT; ++a)
#pragma unroll
    for (int b = 0; b < TE; ++b) {
      float v = acc[a][b];
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) v = v + __shfl_xor(v, o, WAVE);
      if (lane == 0 && t0 + a < T && e0 + b < E) logits[(size_t)(t0 + a) * E + e0 + b] = v;
    }
}

// Order-preserving 64-bit key of (logit, expert): larger key = ranks first
// (logit descending, then index ascending).  -0.0 and +0.0 map to one key.
__device__ __forceinline__ unsigned long long rank_key(float v, int e) {
  uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((unsigned long long)u << 32) | (uint32_t)(0x7fffffff - e);
}

template <int CTRL>
__device__ __forceinline__ unsigned long long dpp_u64(unsigned long long v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xf, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xf, 0xf, false);
  return ((unsigned long long)hi << 32) | lo;
}

// v from the lane DPP control CTRL names, in the rows ROWS selects; other lanes keep v
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned long long dpp_rows_u64(unsigned long long v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)v, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)(v >> 32), (int)(uint32_t)(v >> 32), CTRL,
                                                           ROWS, 0xf, false);
  return ((unsigned long long)hi << 32) | lo;
}

// Maximum over a wavefront whose 64 lanes are all active, all in DPP: within each
// row of 16 lanes (swap neighbours, swap pairs, mirror the half rows, mirror the
// row), then lane 15 of rows 0 and 2 into rows 1 and 3 and lane 31 into rows 2 and
// 3, which leaves the maximum in lane 63; returned to every lane.
__device__ __forceinline__ unsigned long long wave_max_u64(unsigned long long v) {
  unsigned long long w;
  w = dpp_u64<0xb1>(v);  // quad_perm [1,0,3,2]
  v = w > v ? w : v;
  w = dpp_u64<0x4e>(v);  // quad_perm [2,3,0,1]
  v = w > v ? w : v;
  w = dpp_u64<0x141>(v);  // row_half_mirror
  v = w > v ? w : v;
  w = dpp_u64<0x140>(v);  // row_mirror
  v = w > v ? w : v;
  w = dpp_rows_u64<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = w > v ? w : v;
  w = dpp_rows_u64<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  v = w > v ? w : v;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
  return ((unsigned long long)hi << 32) | lo;
}

// The logit a rank key was made from (zero comes back as +0, which the gate
// arithmetic cannot tell from -0).
__device__ __forceinline__ float key_logit(unsigned long long key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// Top-k of one token by one wavefront: k rounds of a wave arg-max over the
// allowed experts (NS per lane), each winner removed; softmax over the k winners.
// Lanes 0..k-1 write the k ids and gates to idx/gates (global or shared memory).
// The logits are loaded together with the mask rather than behind it, and a
// wavefront with two tokens loads both before it selects.
template <int NS>
struct TopkIn {
  float v[NS];
  uint8_t ok[NS];
};

template <int NS>
__device__ __forceinline__ void topk_load(const float* __restrict__ lg, const uint8_t* __restrict__ allowed, int E,
                                          int lane, TopkIn<NS>& in) {
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int e = lane + 64 * s;
    in.v[s] = e < E ? lg[e] : 0.0f;
    in.ok[s] = e < E && (allowed == nullptr || allowed[e] != 0);
  }
}

template <int NS>
__device__ __forceinline__ void topk_pick(const TopkIn<NS>& in, int k, int lane, int32_t* idx, float* gates) {
  unsigned long long key[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) key[s] = in.ok[s] ? rank_key(in.v[s], lane + 64 * s) : 0ull;
  // winner r goes to lane r (value and expert); the largest logit is uniform
  float my_v = 0.0f, top = 0.0f;
  int my_e = -1;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (r < k) {
      unsigned long long b = key[0];
#pragma unroll
      for (int s = 1; s < NS; ++s) b = key[s] > b ? key[s] : b;
      b = wave_max_u64(b);
      if (b != 0ull) {
        const int e = 0x7fffffff - (int)(uint32_t)(b & 0xffffffffu);
#pragma unroll
        for (int s = 0; s < NS; ++s)
          if (lane + 64 * s == e) key[s] = 0ull;
        const float v = key_logit(b);
        if (r == 0) top = v;
        if (lane == r) {
          my_v = v;
          my_e = e;
        }
      }
    }
  }
  // softmax over the k winners, one per lane, summed by a butterfly over 8 lanes
  const float z = (lane < k && my_e >= 0) ? expf(my_v - top) : 0.0f;
  float sum = z;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor(sum, o, WAVE);
  if (lane < k) {
    idx[lane] = my_e;
    gates[lane] = my_e >= 0 ? z / sum : 0.0f;
  }
}

// The same ranks through 32-bit maxima: a round's largest key by DPP maxima, then the least expert that has it by
// ballots, in a third of the instructions.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  const uint32_t w = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xf, false);
  return w > v ? w : v;
}
template <int NS>
__device__ __forceinline__ void topk_pick32(const TopkIn<NS>& in, int k, int lane, int32_t* idx, float* gates) {
  uint32_t key[NS];  // 0: not to be taken; else 1 + the upper word of rank_key (one NaN pattern shares another's)
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const uint32_t u = (uint32_t)(rank_key(in.v[s], 0) >> 32);
    key[s] = in.ok[s] ? (u == 0xffffffffu ? u : u + 1u) : 0u;
  }
  float my_v = 0.0f, top = 0.0f;
  int my_e = -1;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (r < k) {
      uint32_t b = key[0];
#pragma unroll
      for (int s = 1; s < NS; ++s) b = key[s] > b ? key[s] : b;
      b = dpp_umax<0xb1, 0xf>(b);
      b = dpp_umax<0x4e, 0xf>(b);
      b = dpp_umax<0x141, 0xf>(b);
      b = dpp_umax<0x140, 0xf>(b);
      b = dpp_umax<0x142, 0xa>(b);
      b = dpp_umax<0x143, 0xc>(b);
      b = (uint32_t)__builtin_amdgcn_readlane((int)b, 63);
      if (b != 0u) {
        int e = -1;
#pragma unroll
        for (int s = NS - 1; s >= 0; --s) {
          const unsigned long long m = __ballot(key[s] == b);
          if (m) e = 64 * s + __builtin_ctzll(m);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s)
          if (lane + 64 * s == e) key[s] = 0u;
        const float v = key_logit((unsigned long long)(b - 1u) << 32);
        if (r == 0) top = v;
        if (lane == r) {
          my_v = v;
          my_e = e;
        }
      }
    }
  }
  const float z = (lane < k && my_e >= 0) ? expf(my_v - top) : 0.0f;
  float sum = z;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor(sum, o, WAVE);
  if (lane < k) {
    idx[lane] = my_e;
    gates[lane] = my_e >= 0 ? z / sum : 0.0f;
  }
}

// Tokens first, first + step, ... of logits [T, E] by one wavefront, two at a time.
template <int NS>
__device__ __forceinline__ void topk_tokens_ns(const float* __restrict__ logits, const uint8_t* __restrict__ allowed,
                                               int T, int E, int k, int first, int step, int lane, int32_t* idx,
                                               float* gates) {
  for (int t = first; t < T; t += 2 * step) {
    const int t1 = t + step;
    TopkIn<NS> a, b;
    topk_load<NS>(logits + (size_t)t * E, allowed ? allowed + (size_t)t * E : nullptr, E, lane, a);
    if (t1 < T) topk_load<NS>(logits + (size_t)t1 * E, allowed ? allowed + (size_t)t1 * E : nullptr, E, lane, b);
    topk_pick<NS>(a, k, lane, idx + (size_t)t * k, gates + (size_t)t * k);
    if (t1 < T) topk_pick<NS>(b, k, lane, idx + (size_t)t1 * k, gates + (size_t)t1 * k);
  }
}

__device__ __forceinline__ void topk_tokens(const float* __restrict__ logits, const uint8_t* __restrict__ allowed,
                                            int T, int E, int k, int first, int step, int lane, int32_t* idx,
                                            float* gates) {
  if (E <= 64)
    topk_tokens_ns<1>(logits, allowed, T, E, k, first, step, lane, idx, gates);
  else if (E <= 128)
    topk_tokens_ns<2>(logits, allowed, T, E, k, first, step, lane, idx, gates);
  else if (E <= 256)
    topk_tokens_ns<4>(logits, allowed, T, E, k, first, step, lane, idx, gates);
  else if (E <= 512)
    topk_tokens_ns<8>(logits, allowed, T, E, k, first, step, lane, idx, gates);
  else
    topk_tokens_ns<16>(logits, allowed, T, E, k, first, step, lane, idx, gates);
}

}  // namespace dev
}  // namespace ft

// C ABI of the routed layer for a few tokens: argument checks and workspace layout.  See include/ft.h for the
// contract; the kernels are in kernels_moe.hip.
#include <string>

#include "api_checks.h"
#include "internal.h"

using namespace ft;

namespace {

constexpr int32_t kMaxTokens = 64;

size_t record_bytes(const ft_shape* s) { return ft_record_bytes(s); }

// d and d_ff bound the rows that LDS and 32-bit offsets hold.
bool bad_shape(const ft_shape* s) {
  if (!s) return true;
  const size_t S = record_bytes(s);
  return S == 0 || S >= 0x80000000u || s->d > 16384 || s->d_ff > 65536;
}
bool bad_tokens(const ft_shape* s, int32_t T) { return T < 0 || T > kMaxTokens || T * s->k > FT_PLAN_CAP; }

struct Layout {
  size_t logits, grouped, xv, xs, hq, hs, h, part, total;
};
Layout layout(const ft_shape* s, int32_t T) {
  Layout l{};
  const size_t P = (size_t)T * s->k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align256(bytes);
    return o;
  };
  l.logits = take((size_t)T * s->E * 4);
  l.grouped = take(kMoeGroupedBytes);
  if (s->fmt == FT_W_I8) {
    l.xv = take((size_t)T * s->d);
    l.xs = take((size_t)T * 4);
    l.hq = take(P * s->d_ff);
    l.hs = take(P * 4);
    l.h = take(P * s->d_ff * 2);
  } else {
    if (s->fmt == FT_W_MXFP4) l.xv = take((size_t)T * s->d * 2);
    l.h = take(P * s->d_ff * 4);
  }
  const int split = moe_down_split(s->d, s->E);
  if (split > 1) l.part = take((size_t)split * T * s->d * 4);
  l.total = at + 256;
  return l;
}

}  // namespace

extern "C" {

size_t ft_moe_layer_workspace_bytes(const ft_shape* shape, int32_t T) {
  if (bad_shape(shape) || bad_tokens(shape, T)) return 0;
  return layout(shape, T).total;
}

int ft_moe_layer(const ft_shape* shape, const void* x, int32_t T, const void* w_router, const uint8_t* allowed,
                 const void* records, int32_t n_slots, const int32_t* slot_of, const void* residual, void* y,
                 int32_t y_dtype, int32_t* idx, float* gates, void* workspace, size_t workspace_bytes, void* stream) {
  if (bad_shape(shape)) return fail(FT_EINVAL, "moe_layer: bad shape (or a record of 2 GiB, d > 16384, d_ff > 65536)");
  if (bad_tokens(shape, T)) return fail(FT_EINVAL, "moe_layer: T must be 0 .. 64 with T * k <= 512");
  if (y_dtype != FT_T_BF16 && y_dtype != FT_T_FP32) return fail(FT_EINVAL, "moe_layer: y_dtype must be bf16 or fp32");
  if (n_slots < 0 || (!slot_of && n_slots < shape->E))
    return fail(FT_EINVAL, "moe_layer: without slot_of there must be a record for every expert");
  if (T == 0) return FT_OK;
  if (!x || !w_router || (!records && n_slots > 0) || !y || !idx || !gates) return fail(FT_EINVAL, "moe_layer: null pointer");
  const size_t align = y_dtype == FT_T_FP32 ? 4 : 2;
  if (misaligned(x, 16) || misaligned(w_router, 16) || misaligned(records, 16) || misaligned(y, align) ||
      misaligned(residual, align) || misaligned(idx, 4) || misaligned(gates, 4) || misaligned(slot_of, 4))
    return fail(FT_EINVAL, "moe_layer: unaligned pointer");
  if (!workspace || misaligned(workspace, 256)) return fail(FT_EINVAL, "moe_layer: need a 256-byte aligned workspace");
  const Layout l = layout(shape, T);
  if (workspace_bytes < l.total) return fail(FT_ENOMEM, "moe_layer: workspace too small");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeLayer L{};
  L.x = static_cast<const uint16_t*>(x);
  L.w_router = static_cast<const uint16_t*>(w_router);
  L.allowed = allowed;
  L.records = static_cast<const uint8_t*>(records);
  L.n_slots = n_slots;
  L.slot_of = slot_of;
  L.S = record_bytes(shape);
  L.T = T;
  L.d = shape->d;
  L.d_ff = shape->d_ff;
  L.E = shape->E;
  L.k = shape->k;
  L.fmt = shape->fmt;
  L.res = residual;
  L.y = y;
  L.y_f32 = y_dtype == FT_T_FP32;
  L.idx = idx;
  L.gates = gates;
  L.logits = reinterpret_cast<float*>(ws + l.logits);
  L.grouped = ws + l.grouped;
  L.xv = ws + l.xv;
  L.xs = reinterpret_cast<float*>(ws + l.xs);
  L.hq = reinterpret_cast<int8_t*>(ws + l.hq);
  L.hs = reinterpret_cast<float*>(ws + l.hs);
  L.h = ws + l.h;
  L.part = reinterpret_cast<float*>(ws + l.part);
  return launch_moe_layer(L, stream);
}

}  // extern "C"

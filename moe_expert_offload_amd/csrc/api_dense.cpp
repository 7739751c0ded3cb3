// C ABI of the dense operators: argument checks and workspace layout.  See include/ft.h
// for the contract of each call; the kernels are in kernels_dense.hip and kernels_w4.hip.
#include <string>

#include "dense_cut.h"
#include "internal.h"

using ft::fail;

namespace {

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int64_t kMaxLd = 1 << 21;  // a tile's rows stay inside 32-bit byte offsets
// Rows whose tiles' ends, stages and grids (512 threads a tile of 256) stay inside 32 bits.
constexpr int32_t kMaxRows = 0x7fffffff - 511;
bool bad_rows(int32_t T) { return T < 0 || T > kMaxRows; }

bool bad_ld(int64_t ld, int64_t n) { return ld < n || ld > kMaxLd || (ld & 7); }

bool is16(int32_t t) { return t == FT_T_BF16 || t == FT_T_FP16; }
bool is_act(int32_t a) { return a == FT_ACT_SILU || a == FT_ACT_GELU_TANH; }
// (also bounds every row's length by the stride limit)
bool bad_width(int32_t n, int32_t m) { return n <= 0 || n % m || n > kMaxLd / 2; }

// Checks what the forward and backward calls of the block share.
int check_block(const char* fn, int32_t T, int32_t d, int32_t d_ff, int32_t dtype, int32_t act, const void* wg,
                const void* wu, const void* wd, int32_t save_fmt) {
  const std::string f(fn);
  if (bad_rows(T)) return fail(FT_EINVAL, f + ": T must be 0 .. 2^31 - 512");
  if (bad_width(d, 8) || bad_width(d_ff, 8)) return fail(FT_EINVAL, f + ": d and d_ff must be multiples of 8 up to 2^20");
  if (!is16(dtype)) return fail(FT_EINVAL, f + ": dtype must be bf16 or fp16");
  if (!is_act(act)) return fail(FT_EINVAL, f + ": unknown activation");
  if (save_fmt < FT_SAVE_NONE || save_fmt > FT_SAVE_MX8) return fail(FT_EINVAL, f + ": unknown save format");
  if (save_fmt == FT_SAVE_MX8 && d_ff % 32) return fail(FT_EINVAL, f + ": an MX8 save needs d_ff % 32 == 0");
  if (!wg || !wu || !wd) return fail(FT_EINVAL, f + ": null weights");
  if (misaligned(wg, 16) || misaligned(wu, 16) || misaligned(wd, 16)) return fail(FT_EINVAL, f + ": unaligned weights");
  return FT_OK;
}

// Bytes of a block's workspace, with `parts` bytes for the sums of shared tiles.
size_t ffn_bytes(int32_t T, int32_t d_ff, size_t parts) { return align256((size_t)T * d_ff * 2) + parts + 256; }
size_t ffn_bwd_bytes(int32_t T, int32_t d, int32_t d_ff, int32_t save_fmt, bool x_mx8, size_t parts) {
  size_t n = align256((size_t)T * d_ff * 2) + align256((size_t)T * d_ff * 4);  // h; da and du
  if (save_fmt == FT_SAVE_NONE) n += align256((size_t)T * d_ff * 4);           // dh
  if (x_mx8) n += align256((size_t)T * d * 2);                                 // x
  return n + parts + 256;
}

// Points a block at the parts of its saved buffer.
void lay_saved(ft::DenseFfn& F, const void* saved) {
  uint8_t* p = static_cast<uint8_t*>(const_cast<void*>(saved));
  const size_t n = (size_t)F.T * F.d_ff;
  if (F.save_fmt == FT_SAVE_16) {
    F.sa = p;
    F.su = p + 2 * n;
  } else if (F.save_fmt == FT_SAVE_MX8) {
    F.sa = p;
    F.su = p + n;
    F.sca = p + 2 * n;
    F.scu = p + 2 * n + n / 32;
  }
}

// A grid of 512 threads for 16 rows has fewer than 2^32.
constexpr int32_t kMaxW4Rows = (1 << 27) - 16;

int check_w4(const char* fn, const ft_w4_matrix* w) {
  const std::string f(fn);
  if (!w || !w->codes || !w->scales) return fail(FT_EINVAL, f + ": null weights");
  if (w->group != 32 && w->group != 64 && w->group != 128) return fail(FT_EINVAL, f + ": group must be 32, 64 or 128");
  if (w->N <= 0 || w->N > kMaxW4Rows) return fail(FT_EINVAL, f + ": N must be 1 .. 2^27 - 16");
  if (bad_width(w->K, w->group)) return fail(FT_EINVAL, f + ": K must be a multiple of the group, up to 2^20");
  if (misaligned(w->codes, 16) || misaligned(w->scales, 2)) return fail(FT_EINVAL, f + ": unaligned weights");
  return FT_OK;
}

int check_io(const std::string& f, const void* x, int64_t ldx, int64_t K, const void* res, int64_t ldr, const void* y,
             int64_t ldy, int64_t N, int32_t dtype, int32_t y_dtype, size_t align) {
  if (y_dtype != dtype && y_dtype != FT_T_FP32) return fail(FT_EINVAL, f + ": y_dtype must be dtype or fp32");
  if (!x || !y) return fail(FT_EINVAL, f + ": null x or y");
  if (bad_ld(ldx, K)) return fail(FT_EINVAL, f + ": bad row stride of x");
  const bool any = align == 0;  // any stride, the element's alignment
  if (any) align = y_dtype == FT_T_FP32 ? 4 : 2;
  if (any ? ldy < N : bad_ld(ldy, N)) return fail(FT_EINVAL, f + ": bad row stride of y");
  if (res && (any ? ldr < N : bad_ld(ldr, N))) return fail(FT_EINVAL, f + ": bad row stride of residual");
  if (res == y && ldr != ldy) return fail(FT_EINVAL, f + ": a residual in place needs y's stride");
  if (misaligned(x, 16) || misaligned(y, align) || misaligned(res, align))
    return fail(FT_EINVAL, f + ": unaligned pointer");
  return FT_OK;
}

}  // namespace

extern "C" {

size_t ft_gated_ffn_workspace_bytes(int32_t T, int32_t d, int32_t d_ff) {
  if (bad_rows(T) || bad_width(d, 8) || bad_width(d_ff, 8)) return 0;
  return ffn_bytes(T, d_ff, ft::gated_ffn_part_bound(T, d, d_ff, false));
}

size_t ft_gated_ffn_saved_bytes(int32_t T, int32_t d_ff, int32_t save_fmt) {
  if (bad_rows(T) || bad_width(d_ff, 8)) return 0;
  const size_t n = (size_t)T * d_ff;
  if (save_fmt == FT_SAVE_16) return 4 * n;
  if (save_fmt == FT_SAVE_MX8 && d_ff % 32 == 0) return 2 * (n + n / 32);
  return 0;
}

int ft_gated_ffn(const void* x, int64_t ldx, int32_t T, int32_t d, int32_t d_ff, int32_t dtype, int32_t act,
                 const void* w_gate, const void* w_up, const void* w_down, const void* residual, int64_t ldr, void* y,
                 int64_t ldy, int32_t y_dtype, void* saved, int32_t save_fmt, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (int st = check_block("gated_ffn", T, d, d_ff, dtype, act, w_gate, w_up, w_down, save_fmt)) return st;
  if (T == 0) return FT_OK;
  if (int st = check_io("gated_ffn", x, ldx, d, residual, ldr, y, ldy, d, dtype, y_dtype, 16)) return st;
  if (save_fmt != FT_SAVE_NONE && (!saved || misaligned(saved, 16))) return fail(FT_EINVAL, "gated_ffn: bad saved buffer");
  if (!workspace || misaligned(workspace, 256)) return fail(FT_EINVAL, "gated_ffn: need a 256-byte aligned workspace");
  const bool tiles = !ft::gated_ffn_streams(T, save_fmt);
  if (workspace_bytes < ffn_bytes(T, d_ff, tiles ? ft::gated_ffn_part_bytes(T, d, d_ff, false) : 0))
    return fail(FT_ENOMEM, "gated_ffn: workspace too small");
  ft::DenseFfn F{};
  F.x = static_cast<const uint16_t*>(x);
  F.ldx = ldx;
  F.wg = static_cast<const uint16_t*>(w_gate);
  F.wu = static_cast<const uint16_t*>(w_up);
  F.wd = static_cast<const uint16_t*>(w_down);
  F.T = T;
  F.d = d;
  F.d_ff = d_ff;
  F.dtype = dtype;
  F.act = act;
  F.res = residual;
  F.ldr = ldr;
  F.y = y;
  F.ldy = ldy;
  F.y_f32 = y_dtype == FT_T_FP32;
  F.save_fmt = save_fmt;
  lay_saved(F, saved);
  F.h = static_cast<uint16_t*>(workspace);
  F.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256((size_t)T * d_ff * 2));
  return ft::launch_gated_ffn(F, stream);
}

size_t ft_gated_ffn_bwd_workspace_bytes(int32_t T, int32_t d, int32_t d_ff, int32_t save_fmt, int32_t x_mx8) {
  if (bad_rows(T) || bad_width(d, 8) || bad_width(d_ff, 8) || save_fmt < FT_SAVE_NONE || save_fmt > FT_SAVE_MX8) return 0;
  return ffn_bwd_bytes(T, d, d_ff, save_fmt, x_mx8 != 0, ft::gated_ffn_part_bound(T, d, d_ff, true));
}

int ft_gated_ffn_bwd(const void* x, int64_t ldx, const uint8_t* x_scales, int32_t T, int32_t d, int32_t d_ff,
                     int32_t dtype, int32_t act, const void* w_gate, const void* w_up, const void* w_down,
                     const void* saved, int32_t save_fmt, const void* dy, int64_t lddy, void* dx, int64_t lddx,
                     void* dw_gate, void* dw_up, void* dw_down, void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_block("gated_ffn_bwd", T, d, d_ff, dtype, act, w_gate, w_up, w_down, save_fmt)) return st;
  if (!dw_gate != !dw_up || !dw_gate != !dw_down)
    return fail(FT_EINVAL, "gated_ffn_bwd: the weights' gradients are wanted together or not at all");
  if (misaligned(dx, 16) || misaligned(dw_gate, 16) || misaligned(dw_up, 16) || misaligned(dw_down, 16))
    return fail(FT_EINVAL, "gated_ffn_bwd: unaligned gradient");
  if (T > 0) {
    if (!x || !dy || misaligned(x, 16) || misaligned(dy, 16)) return fail(FT_EINVAL, "gated_ffn_bwd: null or unaligned x or dy");
    if (x_scales ? (ldx != d || d % 32) : bad_ld(ldx, d))
      return fail(FT_EINVAL, x_scales ? "gated_ffn_bwd: MX8 x must be contiguous with d % 32 == 0" : "gated_ffn_bwd: bad row stride of x");
    if (bad_ld(lddy, d) || (dx && bad_ld(lddx, d))) return fail(FT_EINVAL, "gated_ffn_bwd: bad row stride of dy or dx");
    if (save_fmt != FT_SAVE_NONE && (!saved || misaligned(saved, 16))) return fail(FT_EINVAL, "gated_ffn_bwd: bad saved buffer");
  }
  if (!workspace || misaligned(workspace, 256)) return fail(FT_EINVAL, "gated_ffn_bwd: need a 256-byte aligned workspace");
  if (workspace_bytes <
      ffn_bwd_bytes(T, d, d_ff, save_fmt, x_scales != nullptr, ft::gated_ffn_part_bytes(T, d, d_ff, true)))
    return fail(FT_ENOMEM, "gated_ffn_bwd: workspace too small");
  if (!dx && !dw_gate) return FT_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto take = [&](size_t bytes) {
    uint8_t* p = ws;
    ws += align256(bytes);
    return p;
  };
  ft::DenseFfn F{};
  F.x = static_cast<const uint16_t*>(x);
  F.ldx = ldx;
  F.wg = static_cast<const uint16_t*>(w_gate);
  F.wu = static_cast<const uint16_t*>(w_up);
  F.wd = static_cast<const uint16_t*>(w_down);
  F.T = T;
  F.d = d;
  F.d_ff = d_ff;
  F.dtype = dtype;
  F.act = act;
  const size_t n = (size_t)T * d_ff;
  F.h = reinterpret_cast<uint16_t*>(take(n * 2));
  ft::DenseGrad G{};
  G.dy = static_cast<const uint16_t*>(dy);
  G.lddy = lddy;
  G.dx = static_cast<uint16_t*>(dx);
  G.lddx = lddx;
  G.dwg = static_cast<uint16_t*>(dw_gate);
  G.dwu = static_cast<uint16_t*>(dw_up);
  G.dwd = static_cast<uint16_t*>(dw_down);
  G.dag = reinterpret_cast<uint16_t*>(take(n * 4));
  F.save_fmt = save_fmt;
  lay_saved(F, saved);
  if (save_fmt == FT_SAVE_NONE) G.dh = reinterpret_cast<float*>(take(n * 4));
  if (x_scales) {
    uint16_t* x16 = reinterpret_cast<uint16_t*>(take((size_t)T * d * 2));
    if (int st = ft::launch_act8_unpack(static_cast<const uint8_t*>(x), x_scales, T, d, dtype == FT_T_FP16, true, x16, d, stream))
      return st;
    F.x = x16;
    F.ldx = d;
  }
  F.part = reinterpret_cast<float*>(ws);
  return ft::launch_gated_ffn_bwd(F, G, stream);
}

int ft_act8_pack(const void* src, int64_t ld, int32_t rows, int32_t n, int32_t dtype, uint8_t* codes, uint8_t* scales,
                 void* stream) {
  if (rows < 0 || bad_width(n, 32)) return fail(FT_EINVAL, "act8_pack: need rows >= 0 and n a multiple of 32");
  if (!is16(dtype)) return fail(FT_EINVAL, "act8_pack: dtype must be bf16 or fp16");
  if (rows == 0) return FT_OK;
  if (bad_ld(ld, n)) return fail(FT_EINVAL, "act8_pack: bad row stride");
  if (!src || !codes || !scales || misaligned(src, 16) || misaligned(codes, 16))
    return fail(FT_EINVAL, "act8_pack: null or unaligned pointer");
  return ft::launch_act8_pack(static_cast<const uint16_t*>(src), ld, rows, n, dtype == FT_T_FP16, codes, scales, stream);
}

int ft_act8_unpack(const uint8_t* codes, const uint8_t* scales, int32_t rows, int32_t n, int32_t dtype, void* dst,
                   int64_t ld, void* stream) {
  if (rows < 0 || bad_width(n, 32)) return fail(FT_EINVAL, "act8_unpack: need rows >= 0 and n a multiple of 32");
  if (!is16(dtype)) return fail(FT_EINVAL, "act8_unpack: dtype must be bf16 or fp16");
  if (rows == 0) return FT_OK;
  if (bad_ld(ld, n)) return fail(FT_EINVAL, "act8_unpack: bad row stride");
  if (!codes || !scales || !dst || misaligned(codes, 16) || misaligned(dst, 16))
    return fail(FT_EINVAL, "act8_unpack: null or unaligned pointer");
  return ft::launch_act8_unpack(codes, scales, rows, n, dtype == FT_T_FP16, false, static_cast<uint16_t*>(dst), ld, stream);
}

int ft_w4_gemv(const void* x, int64_t ldx, int32_t T, int32_t dtype, const ft_w4_matrix* w, const void* residual,
               int64_t ldr, void* y, int64_t ldy, int32_t y_dtype, void* stream) {
  if (int st = check_w4("w4_gemv", w)) return st;
  if (T < 0 || !is16(dtype)) return fail(FT_EINVAL, "w4_gemv: need T >= 0 and bf16 or fp16");
  if (T == 0) return FT_OK;
  if (int st = check_io("w4_gemv", x, ldx, w->K, residual, ldr, y, ldy, w->N, dtype, y_dtype, 0)) return st;
  ft::W4Args A{};
  A.x = static_cast<const uint16_t*>(x);
  A.ldx = ldx;
  A.T = T;
  A.K = w->K;
  A.N = w->N;
  A.G = w->group;
  A.half = dtype == FT_T_FP16;
  A.codes = w->codes;
  A.scales = static_cast<const uint16_t*>(w->scales);
  A.zeros = w->zeros;
  A.res = residual;
  A.ldr = ldr;
  A.y = y;
  A.ldy = ldy;
  A.y_f32 = y_dtype == FT_T_FP32;
  return ft::launch_w4(A, false, stream);
}

size_t ft_w4_gated_ffn_workspace_bytes(int32_t T, int32_t d_ff) {
  if (T < 0 || bad_width(d_ff, 32)) return 0;
  return align256((size_t)T * d_ff * 2) + 256;
}

int ft_w4_gated_ffn(const void* x, int64_t ldx, int32_t T, int32_t dtype, int32_t act, const ft_w4_matrix* gate,
                    const ft_w4_matrix* up, const ft_w4_matrix* down, const void* residual, int64_t ldr, void* y,
                    int64_t ldy, int32_t y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  for (const ft_w4_matrix* w : {gate, up, down})
    if (int st = check_w4("w4_gated_ffn", w)) return st;
  const int d = gate->K, d_ff = gate->N;
  if (up->N != d_ff || up->K != d || down->N != d || down->K != d_ff)
    return fail(FT_EINVAL, "w4_gated_ffn: gate and up must be [d_ff, d] and down [d, d_ff]");
  if (up->group != gate->group) return fail(FT_EINVAL, "w4_gated_ffn: gate and up must have one group size");
  if (T < 0 || !is16(dtype) || !is_act(act)) return fail(FT_EINVAL, "w4_gated_ffn: bad T, dtype or activation");
  if (T == 0) return FT_OK;
  if (int st = check_io("w4_gated_ffn", x, ldx, d, residual, ldr, y, ldy, d, dtype, y_dtype, 0)) return st;
  if (!workspace || misaligned(workspace, 256)) return fail(FT_EINVAL, "w4_gated_ffn: need a 256-byte aligned workspace");
  if (workspace_bytes < ft_w4_gated_ffn_workspace_bytes(T, d_ff)) return fail(FT_ENOMEM, "w4_gated_ffn: workspace too small");
  ft::W4Args A{};
  A.x = static_cast<const uint16_t*>(x);
  A.ldx = ldx;
  A.T = T;
  A.K = d;
  A.N = d_ff;
  A.G = gate->group;
  A.act = act;
  A.half = dtype == FT_T_FP16;
  A.codes = gate->codes;
  A.codes2 = up->codes;
  A.scales = static_cast<const uint16_t*>(gate->scales);
  A.scales2 = static_cast<const uint16_t*>(up->scales);
  A.zeros = gate->zeros;
  A.zeros2 = up->zeros;
  A.h = static_cast<uint16_t*>(workspace);
  if (int st = ft::launch_w4(A, true, stream)) return st;
  ft::W4Args D{};
  D.x = A.h;
  D.ldx = d_ff;
  D.T = T;
  D.K = d_ff;
  D.N = d;
  D.G = down->group;
  D.half = A.half;
  D.codes = down->codes;
  D.scales = static_cast<const uint16_t*>(down->scales);
  D.zeros = down->zeros;
  D.res = residual;
  D.ldr = ldr;
  D.y = y;
  D.ldy = ldy;
  D.y_f32 = y_dtype == FT_T_FP32;
  return ft::launch_w4(D, false, stream);
}

}  // extern "C"

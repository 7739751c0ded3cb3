// C ABI of the products in 8-bit integers: argument checks and workspace layout.  See include/ft.h for the
// contract of each call; the kernels are in kernels_i8.hip.
#include <string>

#include "api_checks.h"
#include "dense_cut.h"
#include "internal.h"

using namespace ft;

namespace {

constexpr int32_t kMaxK = 1 << 16;  // sums of K products of 8-bit integers: at most 2^30 in magnitude
constexpr int32_t kMaxN = (1 << 26) - 256;  // a grid of 1024 threads for 16 channels has fewer than 2^32

// Tiles of 128 x 128 whose grid has fewer than 2^32 threads.
bool too_large(int64_t T, int64_t N) { return ((T + 127) / 128) * ((N + 127) / 128) > (1 << 22); }

bool bad_k(int32_t K) { return K <= 0 || K % 16 || K > kMaxK; }
bool bad_n(int32_t N) { return N <= 0 || N > kMaxN; }

int check_matrix(const char* fn, const ft_i8_matrix* w) {
  const std::string f(fn);
  if (!w || !w->codes || !w->scales) return fail(FT_EINVAL, f + ": null weights");
  if (bad_k(w->K)) return fail(FT_EINVAL, f + ": K must be a multiple of 16 up to 2^16");
  if (bad_n(w->N)) return fail(FT_EINVAL, f + ": N must be 1 .. 2^26 - 256");
  if (misaligned(w->codes, 16) || misaligned(w->scales, 4)) return fail(FT_EINVAL, f + ": unaligned weights");
  return FT_OK;
}

int check_out(const std::string& f, const void* res, int64_t ldr, const void* y, int64_t ldy, int32_t N, int32_t dtype,
              int32_t y_dtype) {
  if (y_dtype != dtype && y_dtype != FT_T_FP32) return fail(FT_EINVAL, f + ": y_dtype must be dtype or fp32");
  if (!y) return fail(FT_EINVAL, f + ": null y");
  if (ldy < N || (res && ldr < N)) return fail(FT_EINVAL, f + ": bad row stride of y or residual");
  if (res == y && ldr != ldy) return fail(FT_EINVAL, f + ": a residual in place needs y's stride");
  const size_t align = y_dtype == FT_T_FP32 ? 4 : 2;
  if (misaligned(y, align) || misaligned(res, align)) return fail(FT_EINVAL, f + ": unaligned pointer");
  return FT_OK;
}

int check_space(const std::string& f, const void* workspace, size_t bytes, size_t need) {
  if (!workspace || misaligned(workspace, 256)) return fail(FT_EINVAL, f + ": need a 256-byte aligned workspace");
  if (bytes < need) return fail(FT_ENOMEM, f + ": workspace too small");
  return FT_OK;
}

I8Mat mat(const ft_i8_matrix* w) { return I8Mat{w->codes, w->scales, w->N, w->K}; }

// Codes and scales of T rows of n.
size_t rows_bytes(int32_t T, int32_t n) { return align256((size_t)T * n) + align256((size_t)T * 4); }

size_t gemm_bytes(int32_t T, int32_t K, bool codes, size_t parts) { return (codes ? 0 : rows_bytes(T, K)) + parts + 256; }
// The two products follow each other: x's codes and h's share a place, and so do their parts.
size_t ffn_bytes(int32_t T, int32_t d, int32_t d_ff, size_t parts) {
  return rows_bytes(T, d > d_ff ? d : d_ff) + align256((size_t)T * d_ff * 2) + parts + 256;
}
size_t larger(size_t a, size_t b) { return a > b ? a : b; }

struct Space {
  uint8_t* at;
  template <class T>
  T* take(size_t bytes) {
    uint8_t* p = at;
    at += align256(bytes);
    return reinterpret_cast<T*>(p);
  }
};

}  // namespace

extern "C" {

int ft_i8_quant(const void* src, int64_t ld, int32_t rows, int32_t n, int32_t dtype, int8_t* codes, float* scales,
                void* stream) {
  if (bad_rows(rows) || bad_k(n)) return fail(FT_EINVAL, "i8_quant: need rows 0 .. 2^31 - 512 and n a multiple of 16 up to 2^16");
  if (!is16(dtype)) return fail(FT_EINVAL, "i8_quant: dtype must be bf16 or fp16");
  if (rows == 0) return FT_OK;
  if (bad_ld(ld, n)) return fail(FT_EINVAL, "i8_quant: bad row stride");
  if (!src || !codes || !scales || misaligned(src, 16) || misaligned(codes, 16) || misaligned(scales, 4))
    return fail(FT_EINVAL, "i8_quant: null or unaligned pointer");
  return launch_i8_quant(static_cast<const uint16_t*>(src), ld, rows, n, dtype == FT_T_FP16, codes, scales, stream);
}

size_t ft_i8_gemm_workspace_bytes(int32_t T, int32_t N, int32_t K, int32_t x_codes) {
  if (bad_rows(T) || bad_n(N) || bad_k(K) || too_large(T, N)) return 0;
  return gemm_bytes(T, K, x_codes != 0, i8_part_bound(T, N, K));
}

int ft_i8_gemm(const void* x, int64_t ldx, const float* x_scales, int32_t T, int32_t dtype, const ft_i8_matrix* w,
               const void* residual, int64_t ldr, void* y, int64_t ldy, int32_t y_dtype, void* workspace,
               size_t workspace_bytes, void* stream) {
  if (int st = check_matrix("i8_gemm", w)) return st;
  if (bad_rows(T) || !is16(dtype)) return fail(FT_EINVAL, "i8_gemm: need T 0 .. 2^31 - 512 and bf16 or fp16");
  if (T == 0) return FT_OK;
  if (too_large(T, w->N)) return fail(FT_EINVAL, "i8_gemm: more than 2^36 results");
  if (!x || misaligned(x, 16) || misaligned(x_scales, 4)) return fail(FT_EINVAL, "i8_gemm: null or unaligned x");
  if (bad_ld(ldx, w->K) || (x_scales && ldx % 16)) return fail(FT_EINVAL, "i8_gemm: bad row stride of x");
  if (int st = check_out("i8_gemm", residual, ldr, y, ldy, w->N, dtype, y_dtype)) return st;
  if (int st = check_space("i8_gemm", workspace, workspace_bytes,
                           gemm_bytes(T, w->K, x_scales != nullptr, i8_part_bytes(T, w->N, w->K))))
    return st;
  const bool half = dtype == FT_T_FP16;
  Space ws{static_cast<uint8_t*>(workspace)};
  I8Rows r{static_cast<const int8_t*>(x), x_scales, ldx, T, nullptr};
  if (!x_scales && i8_own_codes(T, w->K)) {
    r = I8Rows{nullptr, nullptr, ldx, T, static_cast<const uint16_t*>(x)};
  } else if (!x_scales) {
    int8_t* codes = ws.take<int8_t>((size_t)T * w->K);
    float* scales = ws.take<float>((size_t)T * 4);
    if (int st = launch_i8_quant(static_cast<const uint16_t*>(x), ldx, T, w->K, half, codes, scales, stream)) return st;
    r = I8Rows{codes, scales, w->K, T, nullptr};
  }
  return launch_i8_gemm(r, mat(w), I8Out{y, ldy, y_dtype == FT_T_FP32, residual, ldr}, half, ws.take<int>(0), stream);
}

size_t ft_i8_gated_ffn_workspace_bytes(int32_t T, int32_t d, int32_t d_ff) {
  if (bad_rows(T) || bad_k(d) || bad_k(d_ff) || too_large(T, d) || too_large(T, 2 * (int64_t)d_ff)) return 0;
  return ffn_bytes(T, d, d_ff, larger(i8_part_bound(T, 2 * (int64_t)d_ff, d), i8_part_bound(T, d, d_ff)));
}

int ft_i8_gated_ffn(const void* x, int64_t ldx, int32_t T, int32_t dtype, int32_t act, const ft_i8_matrix* gate,
                    const ft_i8_matrix* up, const ft_i8_matrix* down, const void* residual, int64_t ldr, void* y,
                    int64_t ldy, int32_t y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  for (const ft_i8_matrix* w : {gate, up, down})
    if (int st = check_matrix("i8_gated_ffn", w)) return st;
  const int d = gate->K, d_ff = gate->N;
  if (up->N != d_ff || up->K != d || down->N != d || down->K != d_ff)
    return fail(FT_EINVAL, "i8_gated_ffn: gate and up must be [d_ff, d] and down [d, d_ff]");
  if (bad_rows(T) || !is16(dtype) || !is_act(act)) return fail(FT_EINVAL, "i8_gated_ffn: bad T, dtype or activation");
  if (T == 0) return FT_OK;
  if (too_large(T, d) || too_large(T, 2 * (int64_t)d_ff)) return fail(FT_EINVAL, "i8_gated_ffn: more than 2^36 results");
  if (!x || misaligned(x, 16)) return fail(FT_EINVAL, "i8_gated_ffn: null or unaligned x");
  if (bad_ld(ldx, d)) return fail(FT_EINVAL, "i8_gated_ffn: bad row stride of x");
  if (int st = check_out("i8_gated_ffn", residual, ldr, y, ldy, d, dtype, y_dtype)) return st;
  if (int st = check_space("i8_gated_ffn", workspace, workspace_bytes,
                           ffn_bytes(T, d, d_ff, larger(i8_part_bytes(T, 2 * (int64_t)d_ff, d), i8_part_bytes(T, d, d_ff)))))
    return st;
  const bool half = dtype == FT_T_FP16;
  Space ws{static_cast<uint8_t*>(workspace)};
  int8_t* codes = ws.take<int8_t>((size_t)T * (d > d_ff ? d : d_ff));
  float* scales = ws.take<float>((size_t)T * 4);
  uint16_t* h = ws.take<uint16_t>((size_t)T * d_ff * 2);
  int* part = ws.take<int>(0);
  auto rows = [&](const uint16_t* v, int64_t ld, int n, I8Rows& r) -> int {
    if (i8_own_codes(T, n)) {
      r = I8Rows{nullptr, nullptr, ld, T, v};
      return FT_OK;
    }
    r = I8Rows{codes, scales, n, T, nullptr};
    return launch_i8_quant(v, ld, T, n, half, codes, scales, stream);
  };
  I8Rows r;
  if (int st = rows(static_cast<const uint16_t*>(x), ldx, d, r)) return st;
  if (int st = launch_i8_gate_up(r, mat(gate), mat(up), act, h, half, part, stream)) return st;
  if (int st = rows(h, d_ff, d_ff, r)) return st;
  return launch_i8_gemm(r, mat(down), I8Out{y, ldy, y_dtype == FT_T_FP32, residual, ldr}, half, part, stream);
}

}  // extern "C"

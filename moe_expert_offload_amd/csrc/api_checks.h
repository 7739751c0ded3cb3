// Argument checks shared by the stateless operators' entry points (api_dense.cpp, api_i8.cpp, api_moe.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/ft.h"

namespace ft {

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int64_t kMaxLd = 1 << 21;  // a tile's rows stay inside 32-bit byte offsets
// Rows whose tiles' ends, stages and grids (512 threads a tile of 256) stay inside 32 bits.
constexpr int32_t kMaxRows = 0x7fffffff - 511;
inline bool bad_rows(int32_t T) { return T < 0 || T > kMaxRows; }

inline bool bad_ld(int64_t ld, int64_t n) { return ld < n || ld > kMaxLd || (ld & 7); }

inline bool is16(int32_t t) { return t == FT_T_BF16 || t == FT_T_FP16; }
inline bool is_act(int32_t a) { return a == FT_ACT_SILU || a == FT_ACT_GELU_TANH; }
// (also bounds every row's length by the stride limit)
inline bool bad_width(int32_t n, int32_t m) { return n <= 0 || n % m || n > kMaxLd / 2; }

}  // namespace ft

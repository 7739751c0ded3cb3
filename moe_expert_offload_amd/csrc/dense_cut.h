// How the dense operators' tiled products (kernels_dense.hip, kernels_i8.hip) are cut over the compute units, and
// what that takes of a workspace.  Host code, compiled once (dense_cut.cpp): sizes and launches go by the same cut.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/ft.h"

namespace ft {

constexpr int kUnits = 256;  // compute units

// Rows up to which the weights stream once (skinny_kernel); beyond, tiles.
constexpr int kSkinnyRows = 64;
inline bool gated_ffn_streams(int64_t T, int save_fmt) { return T <= kSkinnyRows && save_fmt == FT_SAVE_NONE; }

// How a product is cut.  `n` columns count gate and up apart.
struct Cut {
  int tile;  // 256: 256 x 256; 384: 128 x 256; 128: 128 x 128
  int tiles_m, tiles_n, whole, rest, group, blocks, per, parts;
  size_t part_bytes;
};

Cut cut_of(int64_t M, int64_t n, int stages);  // stages: of 64 k

// What the pieces' sums of a call of T rows take in its tiled form.
size_t gated_ffn_part_bytes(int64_t T, int d, int d_ff, bool backward);
// The most of that over 1 .. T rows, so that a workspace for the largest batch serves every smaller one.
size_t gated_ffn_part_bound(int64_t T, int d, int d_ff, bool backward);

// The same for one product in 8-bit integers, whose stages are 128 k (the same bytes as 64 k of 16 bits).
inline int i8_stages(int K) { return (K + 127) / 128; }
struct I8Cut {
  int tile;   // 0: the weights stream (no tiles); 64: 64 x 128; 128: 128 x 128; 384: 128 x 256; 256: 256 x 256
  bool deep;  // 128 x 128 with three stages in LDS, one tile to a unit
  // `whole` blocks compute a tile each, `parts` further ones `per` stages of the other `rest` tiles, `blocks` to a tile
  int tiles_m, tiles_n, whole, rest, blocks, per, parts;
  size_t part_bytes;
};
I8Cut i8_cut_of(int64_t M, int64_t n, int K);
size_t i8_part_bytes(int64_t T, int64_t n, int K);
size_t i8_part_bound(int64_t T, int64_t n, int K);

}  // namespace ft

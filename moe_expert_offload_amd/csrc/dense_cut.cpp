#include "dense_cut.h"

namespace ft {

// Tiles of 256 columns run one to a compute unit, tiles of 128 x 128 two; both in rounds that cost their
// fullest unit's time, and the last round may share its tiles.  Counted in stages of the 256 x 256 tiles,
// 1.3 us each when the whole chip runs them:
//   a round of 256 x 256 tiles: the stages + 12 (first loads, epilogue); of 128 x 256 tiles: 0.62 of the
//   stages + 9 (M = 1021, N = 5632, K = 2048: 48 us, by 128 x 128 tiles 57);
//   a round of up to 512 tiles of 128 x 128: the stages + 6, of up to 256: half the stages + 5 (M = 1021, N = 2048,
//   K = 11264: 124 us);
//   joining: what a piece writes and the join reads, 0.07 for 256 KB, + 4 (+ 16 behind whole rounds, + 6 for 128 x 128).
// Sharing cuts groups of tiles alike (all into 2 .. 16 parts, or 2 tiles into 3, or 3 into 4), so that blocks
// at the same place of their groups still walk k in step: cutting one line of all tiles into equal
// pieces left M = 2053, N = 4096, K = 11008 at 235 us, as slow as not sharing.
// The constants were fitted at M = 1021, 2053 and 8192 rows. Between 65 and about 500 rows they say too much (65 and
// 128 rows, d = 4096, d_ff = 2048: 50 us for both products, measured 35 and 36), and other cuts have not been timed there.
Cut cut_of(int64_t M, int64_t n, int stages) {
  Cut c{};
  double cost = 1e30;
  for (int mh = 2; mh >= 1; --mh) {
    Cut d{};
    d.tile = mh == 2 ? 256 : 384;
    d.tiles_m = (int)((M + 128 * mh - 1) / (128 * mh));
    d.tiles_n = (int)((n + 255) / 256);
    const int64_t tiles = (int64_t)d.tiles_m * d.tiles_n;
    d.whole = (int)tiles;
    const double stage = mh == 2 ? 1.0 : 0.62, fixed = mh == 2 ? 12 : 9, piece = mh == 2 ? 0.07 : 0.035;
    double t = (double)(tiles / kUnits) * (stage * stages + fixed);
    const int rest = (int)(tiles % kUnits);
    if (rest) {
      double best = stage * stages + fixed;
      auto offer = [&](int group, int blocks) {
        const int groups = (rest + group - 1) / group, per = (group * stages + blocks - 1) / blocks;
        if (groups * blocks > kUnits || per < 4 || per >= stages) return;
        const double u = stage * per + fixed + piece * (groups * blocks + rest) + (tiles > kUnits ? 16 : 4);
        if (u >= best) return;
        best = u;
        d.rest = rest;
        d.whole = (int)tiles - rest;
        d.group = group;
        d.blocks = blocks;
        d.per = per;
        d.parts = groups * blocks;
        d.part_bytes = (size_t)(d.parts + rest) * mh * 128 * 256 * 4;
      };
      for (int k = 2; k <= 16; ++k) offer(1, k);
      offer(2, 3);
      offer(3, 4);
      t += best;
    }
    if (t < cost) {
      cost = t;
      c = d;
    }
  }
  // 128: whole tiles, or all of them cut alike
  const int tm = (int)((M + 127) / 128), tn = (int)((n + 127) / 128);
  const int64_t t128 = (int64_t)tm * tn;
  for (int k = 1; k <= 16; ++k) {
    const int64_t nb = t128 * k, last = nb % (2 * kUnits);
    const int per = (stages + k - 1) / k;
    if (k > 1 && (nb > 2 * kUnits || per < 2)) break;
    double t = (double)(nb / (2 * kUnits)) * (per + 6) + (last == 0 ? 0.0 : last > kUnits ? per + 6 : 0.52 * per + 5);
    if (k > 1) t += 0.0175 * (double)(nb + t128) + 6;
    if (t >= cost) continue;
    cost = t;
    c = Cut{};
    c.tile = 128;
    c.tiles_m = tm;
    c.tiles_n = tn;
    c.whole = c.parts = (int)nb;
    c.blocks = k;
    c.per = per;
    if (k > 1) {
      c.rest = (int)t128;
      c.part_bytes = (size_t)nb * 128 * 128 * 4;
    }
  }
  return c;
}

size_t gated_ffn_part_bytes(int64_t T, int d, int d_ff, bool backward) {
  auto one = [](int64_t M, int64_t n, int64_t K, int segs) { return cut_of(M, n, (int)(segs * ((K + 63) / 64))).part_bytes; };
  size_t m = 0;
  auto up = [&](size_t v) { m = v > m ? v : m; };
  up(one(T, 2 * (int64_t)d_ff, d, 1));
  if (!backward) {
    up(one(T, d, d_ff, 1));
  } else {
    up(one(T, d_ff, d, 1));
    up(one(d, d_ff, T, 1));
    up(one(2 * (int64_t)d_ff, d, T, 1));
    up(one(T, d, d_ff, 2));
  }
  return m;
}

// Rows count by tiles of 128 and, where k runs over them, by stages of 64: every 64th number stands for all (60 us for
// 8192 rows).  Past 16384 rows: what no cut passes, a slot of 256 KB for each unit's piece and each shared tile
// (128 x 128 tiles: 2 kUnits pieces of 64 KB).
template <class Bytes>
static size_t part_bound(int64_t T, Bytes bytes) {
  if (T > 16384) return (size_t)2 * kUnits * (256 << 10);
  size_t m = 0;
  for (int64_t t = 64; t < T + 64; t += 64) {
    const size_t v = bytes(t);
    m = v > m ? v : m;
  }
  return m;
}
size_t gated_ffn_part_bound(int64_t T, int d, int d_ff, bool backward) {
  return part_bound(T, [&](int64_t t) { return gated_ffn_part_bytes(t, d, d_ff, backward); });
}

size_t i8_part_bytes(int64_t T, int64_t n, int K) {
  return T <= kSkinnyRows ? 0 : cut_of(T, n, i8_stages(K)).part_bytes;
}
size_t i8_part_bound(int64_t T, int64_t n, int K) {
  return part_bound(T, [&](int64_t t) { return i8_part_bytes(t, n, K); });
}

}  // namespace ft

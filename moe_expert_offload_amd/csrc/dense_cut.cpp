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

// Products in 8-bit integers.  Each way's time in us, by what was measured from 17 to 8192 rows at (N, K) of (2048, 2048),
// (5632, 2048), (4096, 4096), (11008, 4096) and (4096, 11008): 3 for the launch, and for each round of blocks
//   64 x 128 tiles, two to a unit, three stages in LDS: 0.45 a stage while there is one to a unit, 0.78 for two, + 1.5
//   128 x 128 tiles, two to a unit: 0.85 to 1.1, + 2.5; one to a unit, three stages: 0.64, + 2.2
//   128 x 256 tiles, one to a unit: 0.88, with more than 192 of them up to 1.05, + 2
//   256 x 256 tiles, one to a unit: 1.2, with more than 140 of them up to 1.85 (the clock falls, among other things), + 3
//   joining shared tiles: 4.5, and what the pieces write and the join reads
// against 3 us and the weights at 2.8 (up to 32 rows) or 1.5 TB/s where they stream (up to 64 rows; each 16 channels
// read all tokens' codes, which is what bounds that way).  The best of all ways that were timed is within 10 % of the
// one chosen at three sizes in four.
I8Cut i8_cut_of(int64_t M, int64_t n, int K) {
  const int stages = i8_stages(K);
  I8Cut best{};
  double cost = 1e30;
  if (M <= 16) return best;
  if (M <= kSkinnyRows) cost = 3 + (double)n * K * (M <= 32 ? 0.36e-6 : 0.66e-6);
  auto up = [](double v) { return v > 0 ? v : 0.0; };
  // all tiles shared alike by k blocks, `slots` blocks at once; us(blocks): a stage of a round of so many
  auto even = [&](int tile, bool deep, int bm, int slots, double fixed, double piece, int most, auto us) {
    const int64_t tm = (M + bm - 1) / bm, tn = (n + 127) / 128, tiles = tm * tn;
    for (int k = 1; k <= most; k *= 2) {
      const int per = (stages + k - 1) / k, blocks = (stages + per - 1) / per;
      if (k > 1 && (blocks < k || per < 2 || tiles * blocks > slots)) break;
      const int64_t b = tiles * blocks, last = b % slots;
      double t = 3 + (double)(b / slots) * (us(slots) * per + fixed);
      if (last) t += us((double)last) * per + fixed;
      if (k > 1) t += 4.5 + piece * (double)b;
      if (t >= cost) continue;
      cost = t;
      best = I8Cut{};
      best.tile = tile;
      best.deep = deep;
      best.tiles_m = (int)tm;
      best.tiles_n = (int)tn;
      if (k == 1) {
        best.whole = (int)b;
        continue;
      }
      best.rest = (int)tiles;
      best.blocks = blocks;
      best.per = per;
      best.parts = (int)b;
      best.part_bytes = (size_t)b * bm * 128 * 4;
    }
  };
  even(64, false, 64, 2 * kUnits, 1.5, 0.01, 8, [&](double b) { return b <= 256 ? 0.45 : 0.5 + 0.28 * (b - 256) / 256; });
  even(128, true, 128, kUnits, 2.2, 0.012, 4, [&](double) { return 0.64; });
  even(128, false, 128, 2 * kUnits, 2.5, 0.012, 1, [&](double b) { return 0.85 + 0.25 * up(b - 256) / 256; });
  for (int mh = 1; mh <= 2; ++mh) {
    I8Cut d{};
    d.tile = mh == 2 ? 256 : 384;
    d.tiles_m = (int)((M + 128 * mh - 1) / (128 * mh));
    d.tiles_n = (int)((n + 255) / 256);
    const int64_t tiles = (int64_t)d.tiles_m * d.tiles_n;
    d.whole = (int)tiles;
    const double fixed = mh == 2 ? 3 : 2, piece = mh == 2 ? 0.045 : 0.02;
    auto us = [&](double b) { return mh == 2 ? 1.2 + 0.65 * up(b - 140) / 116 : 0.88 + 0.17 * up(b - 192) / 64; };
    double t = 3 + (double)(tiles / kUnits) * (us(kUnits) * stages + fixed);
    const int rest = (int)(tiles % kUnits);
    if (rest) {
      double last = us(rest) * stages + fixed;
      for (int k = 2; k <= 8; ++k) {
        const int per = (stages + k - 1) / k, blocks = (stages + per - 1) / per;
        if (blocks < k || per < 4 || rest * k > kUnits) continue;
        const double u = us(rest * k) * per + fixed + 4.5 + piece * (rest * k);
        if (u >= last) continue;
        last = u;
        d.rest = rest;
        d.whole = (int)tiles - rest;
        d.blocks = k;
        d.per = per;
        d.parts = rest * k;
        d.part_bytes = (size_t)d.parts * mh * 128 * 256 * 4;
      }
      t += last;
    }
    if (t < cost) {
      cost = t;
      best = d;
    }
  }
  return best;
}

size_t i8_part_bytes(int64_t T, int64_t n, int K) { return i8_cut_of(T, n, K).part_bytes; }
// (between 17 and 64 rows the cut changes at 33 alone)
size_t i8_part_bound(int64_t T, int64_t n, int K) {
  const size_t few = T > 16 ? i8_part_bytes(32, n, K) : 0, all = part_bound(T, [&](int64_t t) { return i8_part_bytes(t, n, K); });
  return few > all ? few : all;
}

}  // namespace ft

"""Cases that reach every way of cutting the products in 8-bit integers.  A way is the tile (64: 64 x 128, 128, 128d:
128 x 128 with three stages in LDS, 384: 128 x 256, 256), then what is shared:
  nothing   whole tiles only
  /k        every tile in k pieces
  +/k       the last round's tiles, behind rounds of whole ones
"stream" has no tiles."""
from tests.dense_cuts import program

# T, N, K, way of the product
GEMM = [
    (1, 8, 16, "stream"), (16, 40, 11008, "stream"), (31, 1000, 304, "stream"), (64, 520, 1104, "stream"),
    (65, 8, 16, "64"), (300, 4096, 4096, "64"), (107, 8, 1936, "64/k"), (64, 4099, 11008, "64/k"), (7032, 1063, 16, "128"),
    (1857, 2066, 768, "128d"), (5303, 8, 4128, "128d/k"), (6530, 521, 16, "384"), (2611, 196, 3232, "384/k"),
    (2137, 7891, 1696, "384+/k"), (7538, 1071, 16, "256"), (743, 5507, 5392, "256/k"), (6254, 2700, 1424, "256+/k"),
]
# T, d, d_ff, ways of gate/up and down
FFN = [
    (1, 16, 16, "stream", "stream"), (33, 256, 784, "stream", "stream"), (65, 16, 16, "64", "64"), (72, 1840, 16, "64/k", "64"),
    (4687, 16, 800, "128", "64"), (7917, 688, 208, "128d", "384"), (5065, 3216, 16, "128d/k", "384"), (6652, 16, 288, "384", "64"),
    (2369, 3472, 80, "384/k", "256"), (2848, 1760, 2864, "384+/k", "384"), (385, 16, 8416, "256", "64/k"),
    (5763, 5376, 368, "256/k", "256"), (1413, 1168, 5712, "256+/k", "64"),
]

_PROGRAM = """
#include <cstdio>
#include "dense_cut.h"
int main() {
  long long M, n, K;
  while (scanf("%lld %lld %lld", &M, &n, &K) == 3) {
    const ft::I8Cut c = ft::i8_cut_of(M, n, (int)K);
    printf("%d %d %d %d %d %d %d %d %zu %d %zu\\n", c.tile, c.tiles_m, c.tiles_n, c.whole, c.rest, c.blocks, c.per,
           c.parts, c.part_bytes, (int)c.deep, ft::i8_part_bound(M, n, (int)K));
  }
}
"""
FIELDS = ("tile", "tiles_m", "tiles_n", "whole", "rest", "blocks", "per", "parts", "part_bytes", "deep", "bound")


def cuts(products, folder):
    """The library's cut of each (M, n, K)."""
    return [dict(zip(FIELDS, v)) for v in program(_PROGRAM, products, folder)]


def way(c):
    if c["tile"] == 0:
        return "stream"
    return f"{c['tile']}{'d' if c['deep'] else ''}" + ("" if not c["rest"] else "+/k" if c["whole"] else "/k")

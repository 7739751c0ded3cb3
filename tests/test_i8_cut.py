"""How the products in 8-bit integers are cut (CPU): every stage of every tile is done once, the sums' slots fit, the size
queries hold for every smaller batch, and the GPU cases reach every way of cutting."""
import random

from tests import i8_cuts as C

WAYS = {"stream", "64", "64/k", "128", "128d", "128d/k", "384", "384/k", "384+/k", "256", "256/k", "256+/k"}
TILES = {64: (64, 128), 128: (128, 128), 384: (128, 256), 256: (256, 256)}


def _check(p, c):
    M, n, K = p
    stages = -(-K // 128)
    if c["tile"] == 0:
        assert M <= 64 and c["part_bytes"] == 0
        return
    bm, bn = TILES[c["tile"]]
    assert M > 16 and c["tiles_m"] == -(-M // bm) and c["tiles_n"] == -(-n // bn)
    assert c["whole"] + c["rest"] == c["tiles_m"] * c["tiles_n"]
    assert (c["whole"] + c["parts"]) * (256 if bn == 128 else 512) < 2 ** 32
    if not c["rest"]:
        assert c["parts"] == 0 and c["part_bytes"] == 0
        return
    assert c["parts"] == c["rest"] * c["blocks"] <= 512
    # pieces [i per, min(stages, (i + 1) per)) of i < blocks: all stages, none empty
    assert (c["blocks"] - 1) * c["per"] < stages <= c["blocks"] * c["per"] and c["blocks"] > 1
    assert c["part_bytes"] == c["parts"] * bm * bn * 4


def test_every_stage_once(tmp_path):
    rng = random.Random(7)
    shapes = [(int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 15)), 16 * int(2 ** rng.uniform(0, 12)))
              for _ in range(6000)] + [(1 << 30, 128, 16), (1 << 22, 8192, 64), (17, 1 << 25, 64), (64, 131072, 65536)]
    shapes += [(T, N, K) for T, N, K, _ in C.GEMM]
    for p, c in zip(shapes, C.cuts(shapes, str(tmp_path))):
        _check(p, c)


def test_bounds_hold_for_smaller_batches(tmp_path):
    rng = random.Random(11)
    for n, K in ((8192, 4096), (4096, 11008), (5632, 2048), (22016, 4096), (512, 65536), (136, 96)):
        Ts = sorted({1, 16, 17, 32, 33, 64, 65, 8192, 16384, 16385, 40000} | {rng.randrange(1, 17000) for _ in range(300)})
        got = C.cuts([(T, n, K) for T in Ts], str(tmp_path))
        assert [c["bound"] for c in got] == sorted(c["bound"] for c in got)
        worst = 0
        for c in got:
            worst = max(worst, c["part_bytes"])
            assert worst <= c["bound"]


def test_cases_reach_every_way(tmp_path):
    got = C.cuts([(T, N, K) for T, N, K, _ in C.GEMM], str(tmp_path))
    assert [C.way(c) for c in got] == [w for *_, w in C.GEMM] and {w for *_, w in C.GEMM} == WAYS
    up = C.cuts([(T, 2 * f, d) for T, d, f, *_ in C.FFN], str(tmp_path))
    down = C.cuts([(T, d, f) for T, d, f, *_ in C.FFN], str(tmp_path))
    assert [(C.way(a), C.way(b)) for a, b in zip(up, down)] == [v[3:] for v in C.FFN]
    assert {v[3] for v in C.FFN} == WAYS

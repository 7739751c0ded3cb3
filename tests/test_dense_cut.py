"""How the dense block's tiled products are cut (CPU): every stage of every tile is done once, the sums' slots fit and
are read as they were written, and the GPU cases reach every way of cutting."""
import random

import pytest
import torch

from tests import dense_cuts as C


def _pieces(c, stages):
    """(tile, first stage, end, slot or -1) of all blocks, as the kernels take them."""
    out = []
    if c["tile"] == 128:
        for b in range(c["parts"]):
            if not c["rest"]:
                out.append((b, 0, stages, -1))
                continue
            t, at = b // c["blocks"], b % c["blocks"] * c["per"]
            out.append((t, at, max(at, min(stages, at + c["per"])), b))
        return out
    out += [(t, 0, stages, -1) for t in range(c["whole"])]
    line = c["group"] * stages
    for b in range(c["parts"] if c["rest"] else 0):
        g = b // c["blocks"]
        at = g * line + (b - g * c["blocks"]) * c["per"]
        end = min(at + c["per"], (g + 1) * line, c["rest"] * stages)
        n = 0
        while at < end:
            t = at // stages
            stop = min(stages, end - t * stages)
            whole = stop - (at - t * stages) == stages
            out.append((c["whole"] + t, at - t * stages, stop, -1 if whole else b + t))
            at, n = t * stages + stop, n + 1
        assert n <= 2
    return out


def _joined(c, t, stages):
    """The slots that the join kernel adds for shared tile t, in order."""
    if c["tile"] == 128:
        return list(range(t * c["blocks"], (t + 1) * c["blocks"]))
    g = t // c["group"]
    at = (t - g * c["group"]) * stages
    first, last = g * c["blocks"] + at // c["per"], g * c["blocks"] + (at + stages - 1) // c["per"]
    return [] if first == last else [b + t for b in range(first, last + 1)]


def test_every_stage_once(tmp_path):
    rng = random.Random(5)
    shapes = [(rng.randrange(1, 9000) if rng.random() < 0.5 else rng.randrange(1, 400), 8 * rng.randrange(1, 2000),
               rng.randrange(0, 300)) for _ in range(4000)]
    shapes += [p[1:] for T, d, f in [v[:3] for v in C.FORWARD + C.BACKWARD] for b in (False, True)
               for p in C.products(T, d, f, b, True)]
    seen = set()
    for (M, n, stages), c in zip(shapes, C.cuts(shapes, str(tmp_path))):
        seen.add(C.way(c))
        bm, bn = {256: (256, 256), 384: (128, 256), 128: (128, 128)}[c["tile"]]
        assert c["tiles_m"] == -(-M // bm) and c["tiles_n"] == -(-n // bn)
        tiles = c["tiles_m"] * c["tiles_n"]
        first_shared = 0 if c["tile"] == 128 and c["rest"] else c["whole"]
        assert tiles == (c["rest"] if first_shared == 0 and c["rest"] else c["whole"] + c["rest"])
        at, slots = {}, {}
        for t, s, e, slot in _pieces(c, stages):
            assert 0 <= t < tiles and 0 <= s <= e <= stages
            if s < e:
                assert at.get(t, 0) == s, "pieces go in the order of k"
                at[t] = e
            if slot >= 0:
                assert slot not in slots and (slot + 1) * bm * bn * 4 <= c["part_bytes"]
                slots[slot] = t
        assert all(at.get(t, 0) == stages for t in range(tiles))
        for t in range(c["rest"]):
            join = _joined(c, t, stages)
            assert sorted(k for k, v in slots.items() if v == first_shared + t) == join
        if c["rest"]:
            assert c["parts"] <= (512 if c["tile"] == 128 else 256)
    assert {"128", "128/k", "256", "256:1/k", "256+1/k", "384", "384:1/k", "384+1/k"} <= seen


def test_sizes_cover_every_smaller_call(tmp_path):
    """What the size queries count for the sums never falls with T and covers each call of T rows."""
    rng = random.Random(6)
    lines, shapes = [], [(4096, 2048), (2048, 768), (4096, 11008), (2048, 5632), (8192, 8), (8, 12312), (264, 11264)]
    for d, f in shapes:
        for T in sorted({rng.randrange(0, 20000) for _ in range(150)} | {0, 1, 64, 65, 128, 129, 16384, 16385, 2 ** 31 - 512}):
            lines += [(T, d, f, b) for b in (0, 1)]
    out = C.program("""
#include <cstdio>
#include "dense_cut.h"
int main() {
  long long T;
  int d, f, b;
  while (scanf("%lld %d %d %d", &T, &d, &f, &b) == 4)
    printf("%zu %zu\\n", ft::gated_ffn_part_bytes(T, d, f, b), ft::gated_ffn_part_bound(T, d, f, b));
}
""", lines, str(tmp_path))
    last = {}
    for (T, d, f, b), (need, bound) in zip(lines, out):
        assert need <= bound and last.get((d, f, b), 0) <= bound, (T, d, f, b)
        last[d, f, b] = bound
        assert T > 0 or need == 0


@pytest.mark.parametrize("cases,backward", [(C.FORWARD, False), (C.BACKWARD, True)])
def test_cases_reach_what_they_are_for(cases, backward, tmp_path):
    names, shapes = [], []
    for i, v in enumerate(cases):
        T, d, f, save = v[0], v[1], v[2], v[5]
        assert backward or save != "none" or T > 64, "fewer rows with nothing kept are not tiled"
        for p in C.products(T, d, f, backward, save == "none"):
            names.append((i, p[0]))
            shapes.append(p[1:])
    got = {}
    for (i, name), c in zip(names, C.cuts(shapes, str(tmp_path))):
        got.setdefault(i, set()).add(f"{name} {C.way(c)}")
    for i, v in enumerate(cases):
        assert set(v[-1].split(", ")) <= got[i], (v, got[i])
    reached = set().union(*(set(v[-1].split(", ")) for v in cases))
    kinds = ["128", "128/k"] + [t + w for t in ("256", "384") for w in ("", ":1/k", ":2/3", ":3/4", "+1/k")]
    for p in ("again", "dh", "dw", "dx") if backward else ("gateup", "out"):
        missing = {f"{p} {k}" for k in kinds} - reached
        assert not missing
    # saves in 8 bits written by whole and shared tiles of each size, and read by each
    eight = set().union(*(got[i] for i, v in enumerate(cases) if v[5] == "mx8"))
    for k in ("128", "256", "256:1/k", "384", "384:1/k" if backward else "384:3/4"):
        assert ("dh " if backward else "gateup ") + k in eight, (k, eight)


# ---- the whole-number cases themselves ---------------------------------------------------

def test_whole_numbers_see_a_lost_share():
    """Inputs as the GPU cases have them: sums exact in fp32, and a result that has lost one stage of 64 k differs in
    most of its elements; one whose pieces are rounded to 16 bits before they are added, in many."""
    T, d, f, dt = 24, 512, 2048, torch.bfloat16
    w = C.Whole(3, "cpu")
    x, wg, wu, wd = w.weights(T, d, f)
    a, u, h, y = C.forward(x, wg, wu, wd, dt)
    assert C.gates_ok(a) and u.abs().max() <= 256 and C.exact_in_fp32(h, wd.t())
    assert torch.equal(torch.nn.functional.silu(a.float()), a.float())
    assert torch.equal(torch.nn.functional.gelu(a.float(), approximate="tanh"), a.float())
    assert torch.equal((h.float() @ wd.float().t()).double(), y)
    for stage in (0, f // 64 - 1):
        lost = C.forward(x, wg, wu, wd, dt, lose=stage)[3]
        assert (C.rounded(lost, torch.float32) != C.rounded(y, torch.float32)).double().mean() > 0.9
        assert (C.rounded(lost, dt) != C.rounded(y, dt)).double().mean() > 0.9
    half = sum(C.rounded(h[:, s] @ wd.t()[s], dt).double() for s in (slice(0, f // 2), slice(f // 2, f)))
    assert (half != y).double().mean() > 0.9
    # a stage of 64 k of a and u themselves
    lost = x.clone()
    lost[:, -64:] = 0
    assert ((lost @ wu.t()) != u).double().mean() > 0.5 and ((lost @ wg.t()) != a).double().mean() > 0.5
    # backward
    dy = w.signs(T, d, p=0.3)
    full, less = (C.backward(x, wg, wu, wd, a, u, dy, dt, lose=s) for s in (None, d // 64 - 1))
    for k in ("dx", "dwg", "dwu"):
        assert (C.rounded(full[k], dt) != C.rounded(less[k], dt)).double().mean() > 0.9, k
    assert C.exact_in_fp32(full["da"], wg) and C.exact_in_fp32(full["du"], wu)
    assert C.exact_in_fp32(full["da"].t(), x) and C.exact_in_fp32(full["du"].t(), x) and C.exact_in_fp32(dy.t(), h)


def test_mx8_of_whole_numbers_is_the_definition():
    from tests import dense_ref as R
    w = C.Whole(4, "cpu")
    v = w.numbers(-500, 500, 40, 64)
    v[3] = 0
    codes, scales = C.mx8(v)
    wc, ws = R.mx8_pack(v)
    assert torch.equal(codes, wc) and torch.equal(scales, ws)

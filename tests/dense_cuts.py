"""Cases that reach every way of cutting the dense block's tiled products, with whole-number inputs whose sums are
exact in fp32, so that the results have one right value each.

A way of cutting is "<product> <tile>": tiles of 128 x 128, 128 x 256 ("384") or 256 x 256, then
  nothing   whole tiles only
  :1/k      every tile's sum over k in 2 .. 16 pieces of its own (128/k: the same of 128 x 128 tiles)
  :2/3 :3/4 two tiles in three pieces, three in four
  +...      the same for the last round's tiles, behind rounds of whole ones
"""
import os
import shutil
import subprocess

import torch

from moe_expert_offload_amd import build

# T, d, f, type, activation, save, residual, type of y, and the ways of cutting that the case is there for
FORWARD = [
    (1, 8, 8, "bf16", "silu", "16", False, "fp32", "gateup 128, out 128"),
    (200, 96, 160, "bf16", "gelu", "mx8", False, "bf16", "gateup 128, out 128"),
    (1, 1160, 1056, "fp16", "gelu", "mx8", True, "fp32", "gateup 128/k, out 128/k"),
    (1, 8224, 4840, "bf16", "silu", "16", True, "bf16", "gateup 384:1/k, out 384:1/k"),
    (8325, 904, 224, "bf16", "silu", "mx8", False, "fp32", "gateup 384, out 256"),
    (8346, 424, 480, "fp16", "silu", "mx8", False, "fp32", "gateup 256, out 384"),
    (143, 6944, 5408, "bf16", "gelu", "mx8", False, "fp32", "gateup 256:1/k, out 384:1/k"),
    (129, 5008, 8344, "bf16", "silu", "16", True, "fp32", "gateup 384:2/3, out 384:1/k"),
    (399, 8328, 5568, "bf16", "silu", "mx8", False, "bf16", "gateup 384:3/4, out 384:2/3"),
    (407, 5552, 8456, "fp16", "silu", "none", True, "fp32", "gateup 256:2/3, out 256:1/k"),
    (666, 1352, 10896, "bf16", "silu", "none", False, "fp32", "gateup 256+1/k, out 384:1/k"),
    (259, 4408, 10944, "bf16", "silu", "mx8", True, "bf16", "gateup 384+1/k, out 384:1/k"),
    (937, 8520, 5632, "bf16", "silu", "16", False, "fp32", "gateup 256:3/4, out 256:2/3"),
    (4998, 3224, 1440, "bf16", "gelu", "none", True, "bf16", "out 256+1/k"),
    (7285, 520, 7584, "bf16", "silu", "none", False, "fp32", "out 384:3/4"),
    (8252, 904, 4768, "fp16", "silu", "16", False, "fp32", "out 384+1/k"),
    (2816, 4096, 11008, "bf16", "silu", "mx8", True, "fp32", "out 256:3/4"),
    (1160, 7504, 9824, "bf16", "silu", "mx8", False, "bf16", "gateup 256+2/3"),
]

# T, d, f, type, activation, save, x in 8 bits, ways
BACKWARD = [
    (1, 416, 12352, "bf16", "silu", "mx8", True, "dh 128, dw 128, dw 256, dx 128/k"),
    (1, 392, 12336, "fp16", "gelu", "none", False, "again 128"),
    (4830, 8224, 8, "bf16", "silu", "none", False, "again 128/k, dh 128/k, dw 128/k, dw 384:1/k, dx 128"),
    (1, 4816, 8200, "bf16", "silu", "none", False, "again 384:1/k, dh 384:1/k, dx 384:1/k"),
    (130, 4832, 8224, "bf16", "silu", "mx8", True, "dh 384:1/k, dx 384:1/k"),
    (4689, 8352, 2080, "bf16", "silu", "mx8", False, "dh 256:3/4"),
    (519, 456, 6752, "bf16", "gelu", "mx8", False, "dh 384, dw 384"),
    (519, 456, 6744, "fp16", "silu", "none", False, "again 256, dh 384, dw 384"),
    (8284, 464, 208, "bf16", "silu", "none", False, "again 384, dx 384"),
    (5890, 1568, 1408, "bf16", "silu", "none", False, "again 256+1/k, dh 256, dw 384:2/3, dx 256"),
    (5890, 1568, 1408, "fp16", "silu", "mx8", True, "dh 256, dw 384:2/3, dx 256"),
    (2198, 7688, 1128, "bf16", "silu", "none", False, "again 384:2/3, dh 256:1/k, dw 256+1/k, dx 256+1/k"),
    (2198, 7680, 1120, "bf16", "silu", "mx8", True, "dh 256:1/k"),
    (134, 8384, 6232, "fp16", "silu", "none", False, "again 256:1/k, dx 256:1/k"),
    (8589, 5392, 456, "bf16", "gelu", "none", False, "again 256:2/3, dh 384:2/3, dw 256:1/k, dw 384:3/4"),
    (773, 4672, 4720, "bf16", "silu", "none", False, "again 384+1/k, dx 384:2/3"),
    (5763, 792, 4160, "bf16", "silu", "16", False, "dw 384+1/k, dx 384:3/4"),
    (944, 8296, 2696, "bf16", "silu", "none", False, "again 384:3/4, dx 384+1/k"),
    (6049, 1296, 3032, "bf16", "gelu", "16", False, "dw 256:2/3, dx 256:2/3"),
    (4638, 8200, 1048, "bf16", "silu", "none", False, "again 256:3/4, dh 384:3/4"),
    (1793, 5528, 4408, "bf16", "silu", "16", False, "dh 384+1/k, dx 256:3/4"),
    (8642, 5408, 944, "fp16", "silu", "16", False, "dh 256:2/3, dw 256:3/4"),
    (1452, 1336, 10992, "bf16", "silu", "16", False, "dh 256+1/k"),
    (8848, 2600, 3840, "bf16", "silu", "16", False, "dx 256+2/3"),
    (7679, 824, 12360, "bf16", "silu", "16", False, "dw 256+2/3"),
]

_PROGRAM = """
#include <cstdio>
#include "dense_cut.h"
int main() {
  long long M, n, stages;
  while (scanf("%lld %lld %lld", &M, &n, &stages) == 3) {
    const ft::Cut c = ft::cut_of(M, n, (int)stages);
    printf("%d %d %d %d %d %d %d %d %d %zu\\n", c.tile, c.tiles_m, c.tiles_n, c.whole, c.rest, c.group, c.blocks, c.per,
           c.parts, c.part_bytes);
  }
}
"""
FIELDS = ("tile", "tiles_m", "tiles_n", "whole", "rest", "group", "blocks", "per", "parts", "part_bytes")


def program(text, lines, folder):
    """The numbers that a program made of the library's own dense_cut prints for each line of numbers."""
    src, exe = os.path.join(folder, "cut.cpp"), os.path.join(folder, "cut")
    with open(src, "w") as f:
        f.write(text)
    cxx = build.CXX if shutil.which(build.CXX) or os.path.exists(build.CXX) else "g++"
    subprocess.run([cxx, "-O1", "-std=c++17", f"-I{build.CSRC}", "-o", exe, src,
                    os.path.join(build.CSRC, "dense_cut.cpp")], check=True, timeout=300)
    lines = "\n".join(" ".join(map(str, p)) for p in lines)
    out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True, timeout=300).stdout
    return [tuple(map(int, v.split())) for v in out.splitlines()]


def cuts(products, folder):
    """The library's cut of each (M, n, stages)."""
    return [dict(zip(FIELDS, v)) for v in program(_PROGRAM, products, folder)]


def products(T, d, f, backward, again):
    """(name, M, n, stages) of the call's products."""
    st = lambda k: (k + 63) // 64  # noqa: E731
    if not backward:
        return [("gateup", T, 2 * f, st(d)), ("out", T, d, st(f))]
    out = [("dh", T, f, st(d)), ("dw", d, f, st(T)), ("dw", 2 * f, d, st(T)), ("dx", T, d, 2 * st(f))]
    return out + ([("again", T, 2 * f, st(d))] if again else [])


def way(c):
    if c["tile"] == 128:
        return "128/k" if c["rest"] else "128"
    if not c["rest"]:
        return str(c["tile"])
    return f"{c['tile']}{'+' if c['whole'] else ':'}{ {1: '1/k', 2: '2/3', 3: '3/4'}[c['group']] }"


# ---- inputs ----------------------------------------------------------------------------

class Whole:
    """Whole-number inputs.  Gates are at least 33, where silu and tanh-gelu are the gate itself and their slope is 1
    to the last bit of fp32 (e^-33 is below half a step of 1), so h = act(a) u, da and du are single products of whole
    numbers: exact in fp32, one rounding to 16 bits.  Weights are -1, 0 or 1 except where they make the gates' level."""

    def __init__(self, seed, on):
        self.g = torch.Generator(device=on).manual_seed(seed)
        self.on = on

    def signs(self, *shape, p):
        """-1, 0 or 1; not 0 with probability p."""
        r = torch.rand(*shape, generator=self.g, device=self.on)
        return (r < p / 2).double() - (r > 1 - p / 2).double()

    def numbers(self, lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=self.g, device=self.on).double()

    def gradient(self, T, d):
        """dy of so few entries that sums over T rows stay below 2^24."""
        return self.signs(T, d, p=min(0.5, 300.0 / T))

    def kept(self, T, f):
        """a and u of a save: gates of 33 .. 223, u of 1 .. 15 with a sign."""
        return self.numbers(33, 223, T, f), self.numbers(1, 15, T, f) * (2 * self.numbers(0, 1, T, f) - 1)

    def kept_mx8(self, T, f):
        """The same in MX8, under scales of 1 and 2: ((codes, scales) of a, those of u)."""
        a = self.numbers(0x61, 0x77, T, f).to(torch.uint8)  # 36 .. 240
        u = self.numbers(1, 8, T, f) * (2 * self.numbers(0, 1, T, f) - 1)
        u = u.float().to(torch.float8_e4m3fn).view(torch.uint8)
        return tuple((c, self.numbers(127, 128, T, f // 32).to(torch.uint8)) for c in (a, u))

    def weights(self, T, d, f, rows=0.5):
        """x, wg, wu, wd: a = x wg^T has mean 128 and spread below 16, u = x wu^T spread below 16."""
        level = max(b for b in (1, 2, 4, 8, 16, 32, 64, 128) if 2 * b <= d)
        p = min(0.5, 200.0 / (rows * d))
        x, wg, wu = self.signs(T, d, p=rows), self.signs(f, d, p=p), self.signs(f, d, p=p)
        x[:, :level] = 1
        wg[:, :level] = 128 // level
        wu[:, :level] = 0
        return x, wg, wu, self.signs(d, f, p=min(0.5, 1500.0 / f))


def exact_in_fp32(v, w):
    """True if no partial sum of v w passes 2^24 (v, w whole numbers)."""
    return (v.abs() @ w.abs()).max().item() < 2 ** 24


def gates_ok(a):
    return 33 <= a.min().item() and a.max().item() <= 256


def rounded(v, dt):
    """Whole numbers below 2^24 (or such times a power of two) to dt, one rounding."""
    return v.float().to(dt)


def _pow2(k):
    """2^k exactly, in 64 bits."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def mx8(v):
    """(codes, scales) of finite fp64 values [rows, n], through torch's conversion to E4M3."""
    b = v.reshape(v.shape[0], -1, 32)
    m, p = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m == 0, torch.full_like(p, -127), torch.where(m <= 0.875, p - 9, p - 8))
    codes = (b * _pow2(-e)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(v.shape), (e + 127).to(torch.uint8).reshape(v.shape[0], -1)


def mx8_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double().reshape(codes.shape[0], -1, 32)
    return (v * _pow2(scales.to(torch.int64) - 127).unsqueeze(-1)).reshape(codes.shape)


def forward(x, wg, wu, wd, dt, residual=None, lose=None):
    """a, u, h (before and after its rounding) and y.  lose: stages of 64 k that a mistaken computation of y would leave
    out."""
    a, u = x @ wg.t(), x @ wu.t()
    h = rounded(a * u, dt).double()
    w = wd.t().clone()
    if lose is not None:
        w[64 * lose:64 * lose + 64] = 0
    y = h @ w
    return a, u, h, y if residual is None else y + residual


def backward(x, wg, wu, wd, a, u, dy, dt, lose=None):
    """h, da, du as rounded and the gradients before their rounding."""
    w = wd.clone()
    if lose is not None:
        w[64 * lose:64 * lose + 64] = 0
    dh = dy @ w
    h, da, du = (rounded(v, dt).double() for v in (a * u, dh * u, dh * a))
    return dict(h=h, da=da, du=du, dx=da @ wg + du @ wu, dwg=da.t() @ x, dwu=du.t() @ x, dwd=dy.t() @ h)

"""Which kernel a bfloat16 product takes (csrc/bf16_tile.h, bf16_few.hip, bf16_grad.hip), read from the
sources, and for every tile of every kind the cheapest shape of a grid that takes it with its ring of stages
run around at least twice."""
import os
import re

import numpy as np

import expert_ffn_amd

_DIR = os.path.join(os.path.dirname(expert_ffn_amd.__file__), "csrc")
_TILE, _GRAD = (open(os.path.join(_DIR, f)).read() for f in ("bf16_tile.h", "bf16_grad.hip"))
f32 = np.float32
KINDS = ("MAT_NT", "MAT_GATED", "MAT_NN", "MAT_TN")


def _table(kind):
    body = _TILE[_TILE.index(f"struct Bf16Tiles<{kind}>"):]
    body = body[:body.index("};\n};")]
    return [(int(a), int(b), *map(f32, c)) for a, b, *c in
            re.findall(r"\{(\d+), (\d+), ([\d.]+)f, ([\d.]+)f, ([\d.]+)f, ([\d.]+)f\}", body)]


TILES = {k: _table(k) for k in KINDS}
# stages and K groups of the tiles in the same order
RINGS = [(int(s), int(g)) for s, g in re.findall(r"return bf16_tile<KIND, AD, \d+, \d+, [^;]*?(\d), (\d)>\(p, s\)", _TILE)]
PAIR = [(int(i), f32(f)) for i, f in re.findall(r"\{(\d), ([\d.]+)f\}", _GRAD[_GRAD.index("PAIR_TILES[]"):].split("};")[0])]
_END = f32(re.search(r"work \+ ([\d.]+)f \* longest", _GRAD).group(1))
_PAIR_RINGS = {int(c): (int(s), int(g)) for c, s, g in re.findall(r"case (\d): return pair<\d+, \d+, \d, \d, (\d), (\d)>", _GRAD)}


def tile_us(c, T, rows, K):
    W = -(-rows // c[0]) * -(-T // c[1])
    steps = f32((K + 63) // 64)
    return c[4] + max(steps * c[2] + c[5], f32((W + 255) // 256) * (steps * c[3] + c[5]))


def pick(kind, T, N, K, adapters=False):
    rows = 2 * N if kind == "MAT_GATED" else N
    tiles = TILES[kind][:11] if adapters else TILES[kind]
    return int(np.argmin([tile_us(c, T, rows, K) for c in tiles]))


def pick_pair(T, N, K):
    """Tile of both gradients of [T, N] . [N, K] in one launch, -1 for one each."""
    best, best_us = -1, tile_us(TILES["MAT_NN"][pick("MAT_NN", T, K, N)], T, K, N) + tile_us(
        TILES["MAT_TN"][pick("MAT_TN", N, K, T)], N, K, T)
    for i, factor in PAIR:
        work = alone = longest = fixed = f32(0)
        for c, (t, n, k) in ((TILES["MAT_NN"][i], (T, K, N)), (TILES["MAT_TN"][i], (N, K, T))):
            steps = f32((k + 63) // 64)
            full = steps * c[3] + c[5]
            work += f32(-(-n // c[0]) * -(-t // c[1])) / f32(256) * full
            alone, longest, fixed = max(alone, steps * c[2] + c[5]), max(longest, full), max(fixed, c[4])
        us = factor * (fixed + max(alone, work + _END * longest))
        if us < best_us:
            best, best_us = i, us
    return best


def wraps(K, ring):
    """Steps of a K group for K elements: enough that every buffer is refilled and read again."""
    stages, groups = ring
    return -(-(-(-K // 64)) // groups) >= 2 * stages + 1


def few_tokens(T, rows, K):
    return T <= 16 or (rows <= 4096 and (T <= 48 or (T <= 64 and K <= 1024)))


_T = (65, 77, 129, 200, 257, 333, 513, 777, 1001, 1500, 2049, 3001, 4097, 6145, 8193)
_N = (72, 200, 333, 520, 1003, 1411, 2051, 2819, 4099, 5635)
_SMALL = (17, 40, 56)
_K = (392, 456, 520, 712, 904, 1160, 1672, 2120)


def shapes(kind, adapters=False):
    """{tile: (T, N, K)}: for NT, GATED T tokens, N channels, K elements; for NN and TN the same sizes of their
    product (rows, columns, contraction)."""
    found = {}
    grid = sorted(((t, n, k) for t in _T for n in _N for k in _K), key=lambda s: s[0] * s[1] * s[2])
    for T, N, K in grid:
        if kind in ("MAT_NN", "MAT_TN"):
            N = N // 8 * 8
        if kind == "MAT_TN":
            T, K = T // 8 * 8, K + 5
        rows = 2 * N if kind == "MAT_GATED" else N
        if kind in ("MAT_NT", "MAT_GATED") and few_tokens(T, rows, K):
            continue
        i = pick(kind, T, N, K, adapters)
        if i not in found and wraps(K, RINGS[i]):
            found[i] = (T, N, K)
    return found


def pair_shapes():
    """{tile: (T, N, K)}, -1: one launch each.  Where a tile has one, a shape whose rings run around in both products."""
    found, any_ = {}, {}
    for T, N, K in sorted(((t, n // 8 * 8, k // 8 * 8) for t in _SMALL + _T for n in _SMALL + _N for k in _SMALL + _N),
                          key=lambda s: s[0] * s[1] * s[2]):
        i = pick_pair(T, N, K)
        any_.setdefault(i, (T, N, K))
        if i < 0 or (wraps(T, _PAIR_RINGS[i]) and wraps(N, _PAIR_RINGS[i])):
            found.setdefault(i, (T, N, K))
    return {**any_, **found}

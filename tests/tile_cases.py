"""Which kernel an 8-bit product takes (csrc/int8.hip: dispatch, pick_tile), read from the source,
and shapes that run every kernel's ring of stages around at least twice."""
import os
import re

import numpy as np

import expert_ffn_amd

_SRC = open(os.path.join(os.path.dirname(expert_ffn_amd.__file__), "csrc", "int8.hip")).read()
# rows of TILES: weight rows, tokens, alone, full, fixed
TILES = [(int(a), int(b), *map(np.float32, (c, d, e)))
         for a, b, c, d, e in re.findall(r"\{(\d+), (\d+), ([\d.]+)f, ([\d.]+)f, ([\d.]+)f\}", _SRC)]
# the template arguments of the tiles in the same order: BN, BT, WN, WT, NSTG, KG
KERNELS = [tuple(map(int, m)) for m in re.findall(r"return tile<(\d+), (\d+), (\d+), (\d+), (\d+), (\d+), GATED>", _SRC)]
_FEW = dict(re.findall(r"(FEW_KG|FEW_NSTG) = (\d+)", _SRC))
FEW_KG, FEW_NSTG = int(_FEW["FEW_KG"]), int(_FEW["FEW_NSTG"])
STEP = 128   # K bytes of a step


def pick_tile(T, rows, K):
    best, best_us = len(TILES) - 1, np.float32(1e30)
    for i, (bn, bt, alone, full, fixed) in enumerate(TILES):
        W = -(-rows // bn) * -(-T // bt)
        if W >= 1 << 22:
            continue
        us = np.float32(-(-K // STEP)) * max(alone, np.float32(-(-W // 256)) * full) + fixed
        if us < best_us:
            best, best_us = i, us
    return best


def few_tokens(T, rows, K):
    """Tiles of 16 tokens of the kernel for few tokens, 0 where a tile kernel runs."""
    few = [(int(t), int(tt), cond) for cond, t, tt in re.findall(
        r"if \((rows <= 256 \* 16 && )?p\.T <= (\d+)[^)]*\) return few<(\d+), GATED>", _SRC)]
    assert few and [tt for _, tt, _ in few] == [1, 2, 3, 4], few
    if T <= 16:
        return 1
    if rows > 256 * 16:
        return 0
    if T <= 48:
        return (T + 15) // 16
    return 4 if T <= 64 and K <= FEW_STEPS_64 * STEP else 0


def kernel_of(T, N, K, gated):
    """(kernel, steps of a K group, stages of its ring)."""
    rows = 2 * N if gated else N
    steps = -(-K // STEP)
    tt = few_tokens(T, rows, K)
    if tt:
        return ("few", tt), -(-steps // FEW_KG), FEW_NSTG
    i = pick_tile(T, rows, K)
    return ("tile", i), -(-steps // KERNELS[i][5]), KERNELS[i][4]


FEW_STEPS_64 = int(re.search(r"p\.T <= 64 && p\.K <= (\d+) \* 128", _SRC).group(1))   # of 49 to 64 tokens

# T, N, K, bf16 output, rows of the output that can be stored in 16-byte pieces; ragged in tokens,
# channels and K
PLAIN = [
    (13, 101, 2832, True, False), (31, 2819, 2832, False, False), (47, 1003, 2832, True, False), (61, 1501, 2800, False, True),
    (67, 131, 3104, False, False), (77, 136, 3216, True, True), (67, 3001, 3104, True, False), (101, 2104, 3104, False, True),
    (67, 4101, 2080, False, False), (67, 4104, 2192, True, True), (67, 3001, 800, True, False), (101, 2056, 912, False, True),
    (67, 8203, 1840, False, False), (67, 8208, 1856, True, True), (201, 8203, 1056, True, False), (201, 8208, 1168, False, True),
    (401, 8203, 800, False, False), (901, 4104, 800, True, True), (701, 8203, 800, True, False), (701, 8208, 912, False, True),
    (901, 8203, 544, False, False), (1601, 5208, 544, True, True), (1601, 8203, 544, True, False), (2601, 5208, 544, False, True),
]
GATED = [
    (13, 101, 2832, True, False), (31, 1003, 2832, False, False), (47, 1003, 2832, True, False), (61, 1501, 2800, False, True),
    (67, 131, 3104, False, False), (77, 136, 3216, True, True), (67, 1503, 3104, True, False), (101, 1104, 3104, False, True),
    (67, 2053, 2080, False, False), (67, 2056, 2192, True, True), (67, 1503, 800, True, False), (101, 1104, 800, False, True),
    (67, 4101, 1840, False, False), (67, 4104, 1856, True, True), (67, 8203, 1056, True, False), (77, 8208, 1168, False, True),
    (131, 8203, 800, False, False), (401, 4104, 800, True, True), (259, 8203, 800, True, False), (519, 5208, 800, False, True),
    (401, 8203, 544, False, False), (901, 4104, 544, True, True), (701, 8203, 544, True, False), (2101, 3008, 544, False, True),
]

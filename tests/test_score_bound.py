"""The error bound of the 32-bit scores that decide between experts (csrc/score.hip,
score_err): its derivation evaluated, and the kernels' arithmetic repeated in numpy with every
exponential off by a whole unit in the adverse direction, against 64 bits."""
import math
import os
import re

import numpy as np
import pytest

import expert_ffn_amd

U = 2.0 ** -24
SOURCE = os.path.join(os.path.dirname(expert_ffn_amd.__file__), "csrc", "score.hip")
F = np.float32


def coefficients():
    m = re.search(r"sigmoid \? ([\d.]+)f \* SU : \(([\d.]+)f \+ ([\d.]+)f \* smax\) \* SU", open(SOURCE).read())
    return tuple(float(v) for v in m.groups())


# experts of a launch, lanes that share a token, experts of a lane at most
KERNELS = [(64, 64, 1), (128, 64, 2), (256, 64, 4), (384, 64, 6), (512, 64, 8),
           (64, 16, 4), (96, 16, 6), (128, 16, 8), (160, 16, 10), (192, 16, 12), (224, 16, 14), (256, 16, 16)]


@pytest.mark.parametrize("E,lanes,per", KERNELS)
def test_derivation(E, lanes, per):
    """(own exponential + sum's exponentials + additions + division and product) s <= (1 + 34 q) U for every q."""
    _, one, per_q = coefficients()
    additions = per - 1 + int(math.log2(lanes))          # a lane's first value is added to 0: exact
    q = np.concatenate([np.geomspace(1.0 / E, 0.5, 20001), 1.0 - np.geomspace(1e-9, 0.5, 20001)])
    mean_x = (1 - q) * np.log(q * (E - 1) / (1 - q))
    log2e = abs(float(F(1.4426950408889634)) / 1.4426950408889634 - 1) / U
    arg = 2 + log2e                                       # difference, product, constant: units of x U
    assert log2e < 0.23
    total = q * (arg * (np.exp(-1.0) + mean_x) + 2 + 2 + additions + 2)
    assert (total <= one + per_q * q).all(), (total - per_q * q).max()
    # sigmoid: s (1 - s) ((1 + constant) x + 2) + the sum's and the division's U of s
    x = np.concatenate([-np.geomspace(1e-6, 80, 20001), np.geomspace(1e-6, 80, 20001)])
    s = 1 / (1 + np.exp(-x))
    assert (s * (1 - s) * ((1 + log2e) * np.abs(x) + 2) + 2 * s).max() <= coefficients()[0]


def rows(E):
    """Logits in fp32: ordinary ones, one large and equal ones, wide ranges, all equal, all but one far below."""
    g = np.random.default_rng(E)
    out = [g.normal(size=(200, E)) * w for w in (0.01, 1, 4, 20)]
    for q in (1.5 / E, 0.05, 0.2, 0.35, 0.6, 0.9, 0.999):
        r = np.full((40, E), math.log((1 - q) / (E - 1)))
        r[:, 0] = math.log(q)
        out.append(r + g.normal(size=(40, 1)) * 30)       # the same scores, other roundings
    out.append(np.zeros((1, E)))
    out.append(np.where(np.arange(E) == E // 2, 0.0, -87.0)[None])
    return np.concatenate(out).astype(F)


def off_by_a_unit(e, way):
    """fp32 exponentials moved by one unit in the last place, up where way > 0."""
    r = e.astype(F)
    return np.where(way > 0, np.nextafter(r, F(np.inf)), np.nextafter(r, F(0)))


def butterfly(v, lanes):
    d = 1
    while d < lanes:
        v = (v + v[:, np.arange(lanes) ^ d]).astype(F)
        d *= 2
    return v[:, :1]


@pytest.mark.parametrize("E,lanes,per", KERNELS)
def test_softmax_scores_in_32_bits(E, lanes, per):
    _, one, per_q = coefficients()
    v = rows(E)
    m = v.max(axis=1, keepdims=True)
    p = np.exp(v.astype(np.float64) - m.astype(np.float64))
    want = p / p.sum(axis=1, keepdims=True)
    arg = ((v - m).astype(F) * F(1.4426950408889634)).astype(F).astype(np.float64)
    e = np.where(v == m, 1.0, np.exp2(arg))
    worst = 0.0
    for way in (1, -1):
        c = np.where(v == m, F(1), off_by_a_unit(e, way))
        full = np.zeros((v.shape[0], lanes * per), F)
        full[:, :E] = c
        s = np.zeros((v.shape[0], lanes), F)
        for i in range(per):
            s = (s + full[:, i * lanes:(i + 1) * lanes]).astype(F)
        inv = (F(1) / butterfly(s, lanes)).astype(F)
        bound = (one + per_q * inv.astype(np.float64)) * U
        # the score's own exponential may be off the other way
        for own in (c, np.where(v == m, F(1), off_by_a_unit(e, -way))):
            err = np.abs((own * inv).astype(F).astype(np.float64) - want) / bound
            worst = max(worst, err.max())
    assert worst <= 1.0, worst


def test_sigmoid_scores_in_32_bits():
    three, _, _ = coefficients()
    g = np.random.default_rng(5)
    v = np.concatenate([g.normal(size=200000) * w for w in (0.1, 2, 20)] + [np.linspace(-100, 88, 100001)]).astype(F)
    want = 1 / (1 + np.exp(-v.astype(np.float64)))
    with np.errstate(over="ignore"):
        e = np.exp2((-v * F(1.4426950408889634)).astype(F).astype(np.float64))
        for way in (1, -1):
            s = (F(1) / (F(1) + off_by_a_unit(e, way)).astype(F)).astype(F)
            assert (np.abs(s.astype(np.float64) - want) <= three * U).all()

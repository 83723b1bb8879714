"""Scored routing on the GPU where its 32-bit choice and its switches can go wrong: near ties
made from the scores themselves, and launches at and beside the thresholds between its kernels."""
import os
import re

import numpy as np
import pytest
import torch

import block_ref as ref
from block_ref import U, f64
from test_gpu_block import BF16, F32, L, close, gen, normal, run_route  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu


def constants():
    """The thresholds of launch_route_score, as the source has them."""
    import expert_ffn_amd
    src = open(os.path.join(os.path.dirname(expert_ffn_amd.__file__), "csrc", "score.hip")).read()
    return {n: int(v) for n, v in re.findall(r"(ROW_\w+) = (\d+)", src)}


def four_tokens_from(E, by_logits):
    """Tokens from which a launch takes the kernel with four tokens to a wave."""
    c = constants()
    return c["ROW_T_LOGITS"] if by_logits else c["ROW_T_SCORES"] + c["ROW_T_SCORES_E"] * E


@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("E,G,keep,top2", [(193, 1, 1, 0), (224, 8, 3, 1), (256, 1, 1, 0), (256, 16, 5, 1), (160, 8, 3, 0),
                                           (512, 1, 1, 0), (384, 12, 4, 1)])
def test_near_ties_from_the_scores(L, E, G, keep, top2, sigmoid):  # noqa: F811
    """A bias that takes nearly all of each score away: c differs from expert to expert by the rounding of the
    bias, below what 32 bits keep of the score.  The choice is that of 64 bits.  With four tokens to a wave up to
    256 experts, else one."""
    g = gen(E + sigmoid)
    T = four_tokens_from(E, False) + 3 if E <= constants()["ROW_E_MAX"] else 300
    base = normal(g, E, scale=2.0)
    base[: E // 8] += 3.0                                  # a few large scores over a long tail
    shift = normal(g, T, 1, scale=8.0) if not sigmoid else torch.zeros(T, 1, device="cuda")
    logits = base + shift                                   # softmax: the same scores but for the logits' rounding
    l0 = f64(base)
    s0 = 1 / (1 + np.exp(-l0)) if sigmoid else np.exp(l0 - l0.max()) / np.exp(l0 - l0.max()).sum()
    bias = torch.from_numpy((0.75 - s0).astype(np.float32)).cuda()
    print(f"[case] near ties T={T} E={E} G={G} sigmoid={sigmoid}", flush=True)
    ids, w = run_route(L, logits, 8, bias=bias, score=sigmoid, n_group=G, topk_group=keep, group_rank=top2)
    want_ids, want_w = ref.route_score(f64(logits), 8, sigmoid, f64(bias), G, keep, top2)
    same = ids == want_ids
    if not same.all():
        l = f64(logits)
        s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max(1, keepdims=True))
        s = s if sigmoid else s / s.sum(1, keepdims=True)
        c = s + f64(bias)
        d = np.abs(np.take_along_axis(c, ids, 1) - np.take_along_axis(c, want_ids, 1))
        # 64-bit scores that agree to a few of their own units may order either way between two programs
        assert (d[~same] <= 2e-15).all(), d.max()
    assert same.mean() > 0.99
    rows = same.all(axis=1)
    close(w[rows], want_w[rows], U * (1 + 1e-6) * np.abs(want_w[rows]) + 1e-45, "weights")


@pytest.mark.parametrize("past", [-1, 0, 1])
@pytest.mark.parametrize("E,k,G,keep,rank,sigmoid,bias,dt", [
    (64, 6, 1, 1, 0, 0, True, F32), (128, 15, 16, 5, 1, 1, True, F32), (192, 12, 3, 2, 1, 0, True, BF16),
    (256, 8, 8, 4, 1, 1, True, F32), (240, 8, 8, 3, 1, 0, False, F32),      # sums of two without a bias: scores
    (256, 8, 1, 1, 0, 0, False, BF16), (100, 5, 10, 4, 0, 1, False, F32),   # logits alone
])
def test_switch_to_four_tokens_by_length(L, E, k, G, keep, rank, sigmoid, bias, dt, past):  # noqa: F811
    """Token counts at and on both sides of the switch."""
    T = four_tokens_from(E, not bias and not rank) + past
    check(L, T, E, k, G, keep, rank, sigmoid, bias, dt)


@pytest.mark.parametrize("E,k,G,keep,rank,sigmoid,bias,dt", [
    (256, 8, 16, 4, 0, 1, True, F32), (256, 8, 32, 4, 0, 1, True, F32),     # groups: the most it takes, and more
    (238, 8, 17, 5, 1, 0, True, BF16), (256, 8, 64, 20, 1, 0, False, F32),
    (128, 15, 1, 1, 0, 0, True, F32), (128, 16, 1, 1, 0, 0, True, F32),     # k likewise
    (256, 9, 1, 1, 0, 1, True, F32), (257, 9, 1, 1, 0, 1, True, F32),       # experts likewise
])
def test_switch_to_four_tokens_by_shape(L, E, k, G, keep, rank, sigmoid, bias, dt):  # noqa: F811
    """Enough tokens for it; the groups, k or experts are the largest it takes, or one more."""
    check(L, four_tokens_from(E, False) + 5, E, k, G, keep, rank, sigmoid, bias, dt)


@pytest.mark.parametrize("by_logits,dt", [(True, BF16), (True, F32), (False, F32)])
@pytest.mark.parametrize("E,G,keep", [(64, 8, 3), (65, 5, 2), (96, 1, 1), (96, 16, 6), (97, 1, 1), (128, 8, 3), (129, 3, 1),
                                      (160, 10, 4), (161, 7, 3), (192, 1, 1), (193, 1, 1), (210, 14, 5), (224, 1, 1),
                                      (224, 16, 7), (225, 15, 4), (256, 1, 1)])
def test_widths_of_four_tokens(L, E, G, keep, by_logits, dt):  # noqa: F811
    """The first and last expert count of each width, by logits and by scores."""
    check(L, four_tokens_from(E, by_logits) + 2, E, 6, G, keep, 0, 0, not by_logits, dt)


def check(L, T, E, k, G, keep, rank, sigmoid, bias, dt):  # noqa: F811
    g = gen(T * 3 + E)
    logits = normal(g, T, E, dtype=dt, scale=1.5)
    b = normal(g, E, scale=0.2) if bias else None
    print(f"[case] route T={T} E={E} k={k} G={G}", flush=True)
    ids, w = run_route(L, logits, k, bias=b, score=sigmoid, n_group=G, topk_group=keep, group_rank=rank, scale=2.5)
    want_ids, want_w = ref.route_score(f64(logits), k, sigmoid, None if b is None else f64(b), G, keep, rank == 1, scale=2.5)
    assert np.array_equal(ids, want_ids)
    # 64-bit arithmetic, one rounding to fp32
    close(w, want_w, U * (1 + 1e-6) * np.abs(want_w) + 1e-45, "weights")

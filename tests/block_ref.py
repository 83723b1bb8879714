"""64-bit reference of the operators around the expert FFN (numpy on the host),
written from their definitions, with the error bounds the tests use.

U = 2^-24 is half a step of fp32 relative to the value; one fp32 operation
errs by at most U of its result.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    """Largest relative error of rounding to dtype (half a step)."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------- routing ----
def route_score(logits, k, sigmoid, bias=None, n_group=1, topk_group=1, top2=False, renorm=True, scale=1.0):
    """ids [T, k] and weights (64 bits) of moe_route_score_topk."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    size = E // n_group
    nan = np.isnan(l)
    low = np.where(nan, -np.inf, l)
    with np.errstate(all="ignore"):
        if sigmoid:
            s = np.where(nan, 0.0, 1.0 / (1.0 + np.exp(-l)))
        else:
            m = low.max(axis=1, keepdims=True)
            e = np.where(nan | (m == -np.inf), 0.0, np.where(l == m, 1.0, np.exp(l - m)))
            tot = e.sum(axis=1, keepdims=True)
            s = np.where(tot > 0, e / tot, 0.0)
        # without a bias the experts' order is that of the logits
        c = l.copy() if bias is None else s + np.asarray(bias, np.float64)[None, :]
        c[nan] = np.nan
        sums = top2 and size > 1             # groups rank by sums of scores
        r = np.where(nan, np.nan, s) if bias is None and sums else c

        def order(v, out=None):
            """Numbers by value, NaN after them, equal ones by index; what is out last."""
            idx = np.broadcast_to(np.arange(v.shape[1]), v.shape)
            return np.lexsort((idx, -np.nan_to_num(v, nan=0.0, posinf=np.inf, neginf=-np.inf), np.isnan(v),
                               np.zeros(v.shape, bool) if out is None else out), axis=1)

        out = np.zeros((T, E), bool)
        if topk_group < n_group:
            g = np.where(np.isnan(r), -np.inf, r).reshape(T, n_group, size)
            g = -np.sort(-g, axis=2)
            rank = g[:, :, 0] + g[:, :, 1] if sums else g[:, :, 0]
            gone = order(rank)[:, topk_group:]
            drop = np.zeros((T, n_group), bool)
            np.put_along_axis(drop, gone, True, axis=1)
            out = np.repeat(drop, size, axis=1)
        ids = order(c, out)[:, :k]
        w = np.take_along_axis(s, ids, axis=1)
        if renorm:
            tot = w.sum(axis=1, keepdims=True)
            w = np.where(tot > 0, w / tot, 0.0)
    return ids.astype(np.int32), w * np.float64(np.float32(scale))


# --------------------------------------------------------------- norms ----
# A sum of squares: at most 32 fused operations in a thread (4 chunks of 8), 6
# lane steps and 16 waves, all terms positive: 54 U of the sum.  r = 1 / sqrt(
# sum / H + eps) halves that and adds the division, the addition, the root and
# the reciprocal: 27 + 1 + 1 + 2.  Then (h r)(off + w): 3 operations.
NORM_U = 40 * U


def norm_in(h, w, off, eps):
    """(x, r) of moe_norm_in in 64 bits; w None: factor 1."""
    h = np.asarray(h, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    f = 1.0 if w is None else np.float64(off) + np.asarray(w, np.float64)
    return h * r * f, r


def codes(u):
    """The code rule in its 32-bit arithmetic: (codes, scale) of fp32 rows u."""
    u = np.asarray(u, np.float32)
    with np.errstate(all="ignore"):
        a = np.abs(u).max(axis=1, keepdims=True)
        s = (a * np.float32(1.0 / 127.0)).astype(np.float32)
        ok = (s > 0) & np.isfinite(s)
        q = np.where(ok, np.clip(np.rint((u / s).astype(np.float32)), -127, 127), 0)
    return q.astype(np.int8), s[:, 0]


def unnormed(h, w, off):
    """u = fl(h * fl(off + w)) in fp32."""
    h = np.asarray(h, np.float32)
    if w is None:
        return h
    return (h * (np.float32(off) + np.asarray(w, np.float32)).astype(np.float32)).astype(np.float32)


def norm_out(h, routes, topk_w, pos, y, w_post, off, eps, gate, block_scale, res_scale):
    """(h_out, bound): h_out in 64 bits before it is rounded to its type, and the
    largest fp32 error of each element."""
    h = np.asarray(h, np.float64)
    T, H = h.shape
    b = np.zeros((T, H))
    a = np.zeros((T, H))          # sum of the magnitudes added
    k = 0
    if routes is not None:
        k = pos.shape[1]
        R = T * k
        for j in range(k):
            live = (pos[:, j] >= 0) & (pos[:, j] < R)
            term = topk_w[live, j].astype(np.float64)[:, None] * routes[pos[live, j]]
            b[live] += term
            a[live] += np.abs(term)
    if y is not None:
        b += y
        a += np.abs(y)
    db = (k + 2) * U * a          # a fused operation per route, one addition for y
    n, dn = b, db
    if w_post is not None:
        r = 1.0 / np.sqrt((b * b).mean(axis=1, keepdims=True) + eps)
        nb = np.sqrt((b * b).sum(axis=1, keepdims=True))
        dr = np.sqrt((db * db).sum(axis=1, keepdims=True)) / np.maximum(nb, 1e-300)   # relative, of r
        dr = np.where(nb > 0, dr, 0.0)
        f = np.float64(off) + np.asarray(w_post, np.float64)
        n = b * r * f
        dn = np.abs(r * f) * (db + np.abs(b) * (dr + NORM_U))
    g = 1.0 if gate is None else np.asarray(gate, np.float64)
    add = block_scale * g * n
    out = res_scale * h + add
    bound = np.abs(block_scale * g) * dn + 3 * U * np.abs(add) + U * np.abs(res_scale * h) + U * np.abs(out) + 1e-37
    return out, bound


# ------------------------------------------------------------- products ----
def matmul_i8(xq, sx, wq, sw, bias=None):
    """(product, bound): acc (exact), then three fp32 roundings and the bias's."""
    acc = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T   # < 2^53: exact
    v = acc * np.asarray(sx, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
    bound = 3.1 * U * np.abs(v)
    if bias is not None:
        v = v + np.asarray(bias, np.float64)[None, :]
        bound = bound + U * np.abs(v)
    return v, bound + 1e-37


def gated(g, u, act):
    """(act(g) u, bound).  act(g) = g / (1 + exp(z)): z carries g's three roundings
    and its polynomial (at most 16 U of |z|), the exponential a step, 1 + e, the
    reciprocal a step, and the two products."""
    z = -g if act == 1 else -2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(all="ignore"):
        v = g / (1.0 + np.exp(z)) * u
    bound = np.abs(v) * (16 * np.abs(z) + 20) * U + 1e-36 * (1.0 + np.abs(g * u))
    return v, bound

"""64-bit reference of the bfloat16 products, their gradients and the low-rank adapters
beside them (torch in double), written from their definitions, and inputs whose sums
are exact.

Whole numbers times a power of two: products and sums below 2^24 units are exact in
fp32 whatever their order, so a 32-bit result equals the 64-bit one and a bfloat16
result is its rounding."""
from __future__ import annotations

import numpy as np
import torch

import block_ref

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def whole(g, *shape, top=2, unit=1.0):
    """Random whole numbers in [-top, top], times `unit` (a power of two), as bf16."""
    v = torch.randint(-top, top + 1, shape, generator=g, device="cuda").float() * unit
    return v.to(BF16)


def adapters(x, ids, a, b, scale, ranks, halves):
    """[T, halves N] in 64 bits: token by token adapter, the low-rank part; and s [T, halves R]."""
    T, n = x.shape[0], b.shape[0]
    R = b.shape[2]
    a = a.view(n, halves, R, x.shape[1])
    N = b.shape[1] // halves
    low = torch.zeros((T, halves * R), dtype=F64, device=x.device)
    out = torch.zeros((T, halves * N), dtype=F64, device=x.device)
    for k in range(n):
        rows = (ids == k).nonzero()[:, 0]
        r = R if ranks is None else min(max(int(ranks[k]), 0), R)
        if not len(rows) or not r:
            continue
        for h in range(halves):
            s = torch.mm(x[rows].to(F64), a[k, h, :r].to(F64).t().contiguous()) * (1.0 if scale is None else scale[k].to(F64))
            low[rows, h * R:h * R + r] = s
            out[rows, h * N:(h + 1) * N] = torch.mm(s, b[k, h * N:(h + 1) * N, :r].to(F64).t().contiguous())
    return low, out


def act_slope(g, act):
    """(act'(g), act(g)) in 64 bits (numpy)."""
    with np.errstate(all="ignore"):
        if act == 1:
            z, dz = g, np.ones_like(g)
        else:
            c = 2.0 * np.sqrt(2.0 / np.pi)
            z, dz = c * (g + 0.044715 * g ** 3), c * (1.0 + 0.134145 * g ** 2)
        q = 1.0 / (1.0 + np.exp(-z))
        return q + g * q * (1.0 - q) * dz, g * q


def gated_grad(pre, dout, act):
    """(dpre, bound) in 64 bits before the rounding to bf16.  The kernel's q = 1 / (1 + e^z) is off by
    e_q = (16 |z| + 4) U of itself (as block_ref.gated derives, without the products), 1 - q by U + e_q q
    absolutely, dz by 5 U; then g q (1 - q) dz three products, a sum, and two products with the gradient."""
    U = block_ref.U
    F = pre.shape[1] // 2
    g, u = pre[:, :F], pre[:, F:]
    slope, value = act_slope(g, act)
    c = 1.0 if act == 1 else 2.0 * np.sqrt(2.0 / np.pi)
    z = g if act == 1 else c * (g + 0.044715 * g ** 3)
    dz = np.ones_like(g) if act == 1 else c * (1.0 + 0.134145 * g ** 2)
    with np.errstate(all="ignore"):
        q = 1.0 / (1.0 + np.exp(-z))
    eq = (16 * np.abs(z) + 4) * U
    t = q * (1 - q)
    dt = t * (eq + 2 * U) + q * (U + eq * q)
    dslope = q * eq + np.abs(g * dz) * (dt + 9 * U * t) + U * (np.abs(slope) + q)
    tiny = 1e-36 * (1 + np.abs(g)) * (1 + np.abs(dz))
    dg, bg = dout * u * slope, np.abs(dout * u) * (dslope + 3 * U * np.abs(slope) + tiny) + 1e-37
    du, bu = dout * value, np.abs(dout) * np.abs(g) * q * (eq + 3 * U) + np.abs(dout * g) * 1e-36 + 1e-37
    return np.concatenate([dg, du], 1), np.concatenate([bg, bu], 1)

"""The bfloat16 products, their backward passes and the low-rank adapters on the GPU against
their 64-bit definitions (bf16_ref.py)."""
import numpy as np
import pytest
import torch

import bf16_ref as ref
import block_ref
from bf16_ref import BF16, F32, F64, whole
from block_ref import f64, half_step
from test_gpu_block import L, check_padding, close, gen, normal, padded  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu
DT = {"f32": F32, "bf16": BF16}


def strided(t, pad=8):
    """The same matrix with rows `pad` elements further apart (NaN between them)."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def equal(got, want, what):
    """got is want (64 bits, exact) rounded to got's type."""
    w = want.to(F32)
    assert (w.to(F64) == want).all(), "the test's sums are not exact"
    w = w.to(got.dtype)
    if not torch.equal(got, w):
        bad = got != w
        at = bad.nonzero()[:5].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {at}")


# T, N, K, type, pad of the output's rows: few tokens, every tile, ragged tokens, channels and K
PLAIN = [
    (1, 1, 8, "f32", 0), (1, 2816, 2112, "bf16", 0), (2, 17, 64, "f32", 3), (5, 100, 72, "bf16", 1), (16, 4099, 136, "f32", 0),
    (17, 4097, 200, "bf16", 8), (31, 2112, 1424, "bf16", 0), (33, 333, 520, "f32", 5), (48, 4096, 64, "bf16", 0),
    (49, 77, 1000, "f32", 1), (64, 4100, 328, "bf16", 4), (65, 1411, 1424, "f32", 1), (77, 2819, 704, "bf16", 5),
    (129, 2816, 2112, "bf16", 0), (200, 333, 4096, "f32", 0), (255, 1000, 264, "bf16", 0), (257, 4096, 72, "f32", 2),
    (512, 2816, 704, "bf16", 0), (1000, 1023, 520, "f32", 1), (1024, 4224, 192, "bf16", 0), (2049, 2817, 264, "bf16", 1),
    (3000, 5632, 136, "f32", 0), (4100, 4104, 328, "bf16", 0), (8193, 300, 64, "f32", 4),
]


@pytest.mark.parametrize("T,N,K,dt,pad", PLAIN)
def test_matmul(L, T, N, K, dt, pad):  # noqa: F811
    print(f"[case] matmul_bf16 T={T} N={N} K={K} {dt}", flush=True)
    g = gen(T + 3 * N + K)
    x, w = strided(whole(g, T, K)), strided(whole(g, N, K, top=3), 16)
    out, buf = padded(T, N, DT[dt], pad, 2.0)
    L.matmul_bf16(x, w, out)
    torch.cuda.synchronize()
    check_padding(buf, N, 2.0)
    equal(out, x.to(F64) @ w.to(F64).t().contiguous(), "out")


# T, F, K, act, type, pre
GATED = [
    (1, 1, 8, 0, "f32", True), (1, 2112, 2816, 0, "bf16", False), (3, 100, 72, 1, "bf16", True), (16, 2051, 136, 1, "f32", False),
    (17, 704, 1424, 0, "bf16", True), (40, 1411, 264, 1, "f32", True), (48, 2048, 64, 0, "bf16", False),
    (64, 100, 2112, 1, "bf16", True), (77, 1411, 1424, 1, "f32", False), (129, 2112, 264, 0, "bf16", True),
    (255, 77, 1000, 1, "f32", True), (300, 1000, 520, 0, "bf16", False), (513, 2112, 328, 1, "bf16", True),
    (1024, 2112, 264, 0, "bf16", False), (2047, 1409, 136, 1, "bf16", True), (4096, 2112, 72, 0, "f32", True),
    (4097, 4099, 200, 1, "bf16", True),
]


@pytest.mark.parametrize("T,F,K,act,dt,pre", GATED)
def test_gated(L, T, F, K, act, dt, pre):  # noqa: F811
    print(f"[case] gated_matmul_bf16 T={T} F={F} K={K} act={act} {dt} pre={pre}", flush=True)
    g = gen(T + 3 * F + K)
    # sums with 2^-6 units of order 1 to 3
    unit = 2.0 ** -round(np.log2(max(2.0, 2.0 * K ** 0.5)))
    x, w = strided(whole(g, T, K)), strided(whole(g, 2 * F, K, unit=unit), 16)
    out, buf = padded(T, F, DT[dt], 1 if F % 2 else 8, 2.0)
    p, pbuf = padded(T, 2 * F, BF16, 3, 2.0) if pre else (None, None)
    L.gated_matmul_bf16(x, w, act, out, pre=p)
    torch.cuda.synchronize()
    check_padding(buf, F, 2.0)
    v = x.to(F64) @ w.to(F64).t().contiguous()
    if pre:
        check_padding(pbuf, 2 * F, 2.0)
        equal(p, v, "pre")
    v = v.cpu().numpy()
    want, bound = block_ref.gated(v[:, :F], v[:, F:], act)
    close(f64(out), want, bound + half_step(out.dtype) * (abs(want) + bound), "out")


# T, N, K
GRAD = [
    (1, 8, 8), (1, 2816, 704), (3, 72, 200), (16, 2112, 264), (33, 704, 1424), (64, 64, 64), (65, 520, 136), (77, 1000, 712),
    (129, 2816, 328), (200, 72, 2816), (333, 1408, 1424), (513, 4096, 264), (1001, 2816, 704), (1024, 264, 4096),
    (2049, 712, 520), (4096, 1024, 2112), (5000, 328, 328), (8200, 64, 136),
]


@pytest.mark.parametrize("T,N,K", GRAD)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_matmul_backward(L, T, N, K, dt):  # noqa: F811
    print(f"[case] matmul_bf16_backward T={T} N={N} K={K} {dt}", flush=True)
    g = gen(T + 3 * N + K)
    x, w, d = strided(whole(g, T, K)), strided(whole(g, N, K), 24), strided(whole(g, T, N), 16)
    dx, xbuf = padded(T, K, DT[dt], 8, 2.0)
    dw, wbuf = padded(N, K, DT[dt], 3, 2.0)
    L.matmul_bf16_backward(x, w, d, dx=dx, dw=dw)
    torch.cuda.synchronize()
    check_padding(xbuf, K, 2.0)
    check_padding(wbuf, K, 2.0)
    equal(dx, d.to(F64) @ w.to(F64).contiguous(), "dx")
    equal(dw, d.to(F64).t().contiguous() @ x.to(F64).contiguous(), "dw")


@pytest.mark.parametrize("T,F,K,act,inplace", [(1, 8, 8, 0, False), (5, 72, 136, 1, True), (77, 704, 1424, 1, False),
                                               (333, 1408, 264, 0, True), (1030, 2112, 328, 0, False), (2049, 264, 712, 1, False)])
def test_gated_backward(L, T, F, K, act, inplace):  # noqa: F811
    print(f"[case] gated_matmul_bf16_backward T={T} F={F} K={K} act={act}", flush=True)
    g = gen(T + 3 * F + K)
    x, w = strided(normal(g, T, K, dtype=BF16)), strided(normal(g, 2 * F, K, dtype=BF16, scale=K ** -0.5), 16)
    pre, d = strided(normal(g, T, 2 * F, dtype=BF16, scale=2.0), 16), strided(normal(g, T, F, dtype=BF16))
    want, bound = ref.gated_grad(f64(pre), f64(d), act)
    dp, pbuf = padded(T, 2 * F, BF16, 8, 2.0)
    if inplace:
        dp = pre
    dx, xbuf = padded(T, K, F32, 1, 2.0)
    dw, wbuf = padded(2 * F, K, F32, 8, 2.0)
    L.gated_matmul_bf16_backward(x, w, act, pre, d, dp, dx=dx, dw=dw)
    torch.cuda.synchronize()
    if not inplace:
        check_padding(pbuf, 2 * F, 2.0)
    check_padding(xbuf, K, 2.0)
    check_padding(wbuf, K, 2.0)
    # a value near the smallest normal number may be flushed to zero
    close(f64(dp), want, bound + half_step(BF16) * (abs(want) + bound) + 2.0 ** -126, "dpre")
    # dx and dw are those of the rounded dpre.  A sum of n products: every addition, and every product the
    # matrix unit holds, errs by at most two half steps of the sum of the magnitudes so far
    a, b, c = dp.to(F64).contiguous(), w.to(F64).contiguous(), x.to(F64).contiguous()
    at = a.t().contiguous()
    for got, want, mag, n, what in ((dx, a @ b, a.abs() @ b.abs(), 2 * F, "dx"), (dw, at @ c, at.abs() @ c.abs(), T, "dw")):
        close(f64(got), f64(want), f64(mag) * 2 * (n + 8) * block_ref.U, what)


def test_gated_backward_against_differences(L):  # noqa: F811
    """The whole backward pass against central differences of the 64-bit forward pass, in a direction of
    every input: the directional derivative is sum(dout * d out)."""
    T, F, K = 37, 104, 136
    for act in (0, 1):
        g = gen(act)
        x, w = normal(g, T, K, dtype=BF16), normal(g, 2 * F, K, dtype=BF16, scale=K ** -0.5)
        pre, out = torch.empty(T, 2 * F, dtype=BF16, device="cuda"), torch.empty(T, F, dtype=BF16, device="cuda")
        L.gated_matmul_bf16(x, w, act, out, pre=pre)
        d = normal(g, T, F, dtype=BF16)
        dx, dw = torch.empty(T, K, device="cuda"), torch.empty(2 * F, K, device="cuda")
        L.gated_matmul_bf16_backward(x, w, act, pre, d, torch.empty_like(pre), dx=dx, dw=dw)
        vx, vw = normal(g, T, K).double(), normal(g, 2 * F, K).double()

        def loss(e):
            v = (x.double() + e * vx) @ (w.double() + e * vw).t().contiguous()
            return (torch.from_numpy(ref.act_slope(f64(v[:, :F]), act)[1]).cuda() * v[:, F:] * d.double()).sum()

        h = 2.0 ** -12
        want = (loss(h) - loss(-h)) / (2 * h)
        got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
        # terms are off by their roundings to bf16 (pre twice, dpre once: at most 3 half steps of slopes of
        # order 1), which are independent and of either sign: 6 standard deviations of their sum
        spread = 3 * half_step(BF16) * float(((dx.double() * vx).square().sum() + (dw.double() * vw).square().sum()).sqrt())
        assert abs(float(got - want)) <= 6 * spread, (act, float(got), float(want), spread)


def make_adapters(g, T, K, N, n, R, halves, kind):
    """x sparse in [-1, 1] and whole numbers throughout, so that s and the products are exact."""
    x = (whole(g, T, K, top=1).float() * (torch.rand((T, K), generator=g, device="cuda") < min(1.0, 200 / K))).to(BF16)
    a, b = whole(g, n, halves, R, K, top=1), whole(g, n, halves * N, R, top=2)
    w = whole(g, halves * N, K, top=2)
    if kind == "tokens":
        ids = torch.randint(-1, n, (T,), generator=g, device="cuda")
    elif kind == "runs":
        ids = torch.randint(-1, n, (T // 100 + 1,), generator=g, device="cuda").repeat_interleave(100)[:T]
    elif kind == "none":
        ids = torch.where(torch.arange(T, device="cuda") % 2 == 0, -1, n)      # outside on both sides
    else:
        ids = torch.full((T,), n - 1, device="cuda")
    scale = 2.0 ** torch.randint(-1, 2, (n,), generator=g, device="cuda").float()
    return x, w, a, b, ids.to(torch.int32).contiguous(), scale


# T, N, K, n, R, gated, ids, ranks
ADAPTERS = [
    (1, 17, 64, 1, 8, False, "one", False), (1, 2816, 2112, 8, 16, False, "tokens", False), (7, 100, 72, 5, 24, False, "tokens", True),
    (16, 2112, 2816, 32, 16, True, "tokens", False), (16, 333, 200, 40, 40, False, "tokens", True), (16, 333, 200, 4, 8, True, "none", False),
    (17, 700, 136, 3, 72, True, "tokens", True), (48, 2048, 264, 64, 16, False, "tokens", True), (47, 1411, 520, 9, 8, True, "one", True),
    (64, 4200, 264, 7, 16, False, "tokens", False), (65, 2112, 704, 64, 64, True, "tokens", True), (129, 2816, 2112, 32, 64, False, "tokens", True),
    (200, 1003, 136, 300, 16, False, "tokens", True), (257, 4096, 328, 4, 128, True, "runs", False), (300, 77, 1000, 6, 56, False, "runs", True),
    (512, 520, 264, 3, 16, False, "none", True), (1000, 2112, 520, 24, 32, True, "runs", True), (1024, 2816, 264, 16, 16, False, "runs", False),
    (2049, 1409, 200, 64, 8, True, "tokens", False), (2100, 4099, 136, 2, 256, False, "runs", True), (4096, 2112, 72, 24, 32, True, "runs", True),
]


@pytest.mark.parametrize("T,N,K,n,R,gated,kind,uneven", ADAPTERS)
def test_adapters(L, T, N, K, n, R, gated, kind, uneven):  # noqa: F811
    print(f"[case] adapters T={T} N={N} K={K} n={n} R={R} gated={gated} {kind} uneven={uneven}", flush=True)
    g = gen(T + 3 * N + K + 7 * R)
    halves = 2 if gated else 1
    x, w, a, b, ids, scale = make_adapters(g, T, K, N, n, R, halves, kind)
    ranks = None
    if uneven:   # from none to more than R
        ranks = torch.randint(-1, R + 3, (n,), generator=g, device="cuda", dtype=torch.int32)
    low, up = ref.adapters(x, ids, a, b, scale, ranks, halves)
    assert low.abs().max() <= 256
    if uneven:   # what lies past a rank is not used
        past = torch.arange(R, device="cuda")[None, :] >= ranks[:, None]
        a = torch.where(past[:, None, :, None], torch.full_like(a, float("nan")), a)
        b = torch.where(past[:, None, :], torch.full_like(b, float("inf")), b)
    s, sbuf = padded(T, halves * R, BF16, 8, 2.0)
    L.adapter_shrink(strided(x), ids, a if gated else a[:, 0], scale, s, ranks=ranks)
    torch.cuda.synchronize()
    check_padding(sbuf, halves * R, 2.0)
    equal(s, low, "s")
    v = x.to(F64) @ w.to(F64).t().contiguous() + up
    if not gated:
        out, buf = padded(T, N, F32, 3, 2.0)
        L.matmul_bf16(x, w, out, s=s, adapter_ids=ids, b=b, ranks=ranks)
        torch.cuda.synchronize()
        check_padding(buf, N, 2.0)
        equal(out, v, "out")
        return
    out, buf = padded(T, N, F32, 3, 2.0)
    pre, pbuf = padded(T, 2 * N, BF16, 1, 2.0)
    L.gated_matmul_bf16(x, w, 1, out, pre=pre, s=s, adapter_ids=ids, b=b, ranks=ranks)
    torch.cuda.synchronize()
    check_padding(buf, N, 2.0)
    check_padding(pbuf, 2 * N, 2.0)
    equal(pre, v, "pre")
    v = v.cpu().numpy()
    want, bound = block_ref.gated(v[:, :N], v[:, N:], 1)
    close(f64(out), want, bound, "out")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_backward_of_no_tokens(L, dt):  # noqa: F811
    """The weights' gradient of no tokens is zeros; the rows' has no rows."""
    N, K = 112, 72
    x, d, w = torch.empty(0, K, dtype=BF16, device="cuda"), torch.empty(0, N, dtype=BF16, device="cuda"), whole(gen(1), N, K)
    dw, buf = padded(N, K, DT[dt], 8, 2.0)
    L.matmul_bf16_backward(x, w, d, dx=torch.empty(0, K, device="cuda"), dw=dw)
    torch.cuda.synchronize()
    check_padding(buf, K, 2.0)
    assert (dw == 0).all()
    L.matmul_bf16_backward(x, w, d, dx=torch.empty(0, K, device="cuda"))
    dw.fill_(3.0)
    g = d[:, :N // 2]
    L.gated_matmul_bf16_backward(x, w, 0, d, g, torch.empty_like(d), dw=dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


@pytest.mark.parametrize("T,N,K", GRAD)
def test_one_gradient_is_that_of_both(L, T, N, K):  # noqa: F811
    """dx and dw asked for apart (a launch each) and together (one launch for small shapes): exact sums."""
    g = gen(T + 5 * N + K)
    x, w, d = whole(g, T, K), whole(g, N, K), whole(g, T, N)
    out = [torch.full((r, K), 7.0, dtype=BF16, device="cuda") for r in (T, N, T, N)]
    L.matmul_bf16_backward(x, w, d, dx=out[0], dw=out[1])
    L.matmul_bf16_backward(x, w, d, dx=out[2])
    L.matmul_bf16_backward(x, w, d, dw=out[3])
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    equal(out[0], d.to(F64) @ w.to(F64).contiguous(), "dx")

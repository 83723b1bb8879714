"""The operators around the expert FFN on the GPU against their 64-bit
definitions (block_ref.py): scored routing, the norms before and after the block,
the activation codes and the 8-bit products."""
import numpy as np
import pytest
import torch

import block_ref as ref
from block_ref import U, f64, half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def L():
    import expert_ffn_amd as lib
    lib.lib()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def padded(rows, cols, dtype, pad, fill):
    """A view of rows x cols inside a larger buffer full of `fill`, and the buffer."""
    buf = torch.full((rows + 2, cols + pad), fill, dtype=dtype, device="cuda")
    return buf[1:rows + 1, :cols], buf


def check_padding(buf, cols, fill):
    assert (buf[0] == fill).all() and (buf[-1] == fill).all(), "rows beside the output were written"
    assert (buf[:, cols:] == fill).all(), "columns beside the output were written"


def close(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    bad = ~(np.abs(got - want) <= bound)
    bad &= ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} elements off, worst "
                           f"{np.nanmax(np.abs(got - want) / np.maximum(bound, 1e-300)):.3g} x the bound")


# ------------------------------------------------------------- routing ----
def run_route(L, logits, k, bias=None, **kw):
    T = logits.shape[0]
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    L.route_score_topk(logits, k, ids[:T], w[:T], bias=bias, **kw)
    torch.cuda.synchronize()
    assert (ids[T] == -7).all() and (w[T] == -7).all()
    return ids[:T].cpu().numpy(), f64(w[:T])


@pytest.mark.parametrize("T,E,k,G,keep,rank,sigmoid,bias,dt,scale,renorm", [
    (1, 1, 1, 1, 1, 0, 0, False, F32, 1.0, 1),
    (1, 128, 8, 1, 1, 0, 0, True, F32, 1.0, 1),
    (16, 128, 8, 1, 1, 0, 0, False, F32, 1.0, 0),
    (5, 7, 7, 1, 1, 0, 1, True, F32, 2.5, 1),
    (67, 256, 8, 8, 4, 1, 1, True, F32, 2.5, 1),
    (66, 256, 8, 8, 4, 1, 0, True, BF16, 1.0, 1),
    (33, 160, 6, 8, 3, 0, 0, False, BF16, 16.0, 0),
    (19, 512, 32, 64, 5, 1, 1, True, F32, 1.0, 1),
    (19, 64, 2, 64, 7, 1, 1, True, F32, 1.0, 1),      # groups of one expert
    (21, 192, 12, 3, 2, 1, 0, False, F32, 1.0, 1),
    (9, 90, 9, 10, 1, 0, 1, True, F32, 1.0, 0),       # k = the kept group's size
    (130, 100, 4, 1, 1, 0, 1, False, F32, 1.0, 1),
    (37, 384, 8, 1, 1, 0, 1, True, BF16, 1.0, 1),
    (17, 257, 9, 1, 1, 0, 0, True, F32, 1.0, 1),
    # four tokens to a wave: every width, ragged token counts, the largest k and group count it takes
    (4099, 160, 6, 8, 3, 0, 0, False, BF16, 1.0, 1),
    (4097, 61, 15, 1, 1, 0, 1, False, F32, 1.0, 0),
    (4096, 128, 8, 16, 5, 0, 0, False, F32, 2.5, 0),
    (12289, 256, 8, 8, 4, 1, 1, True, F32, 2.5, 1),
    (12290, 192, 12, 3, 2, 1, 0, True, BF16, 1.0, 1),
    (12291, 48, 3, 16, 7, 1, 0, True, F32, 1.0, 0),
    (12292, 100, 15, 1, 1, 0, 1, True, F32, 1.0, 1),
    (12300, 256, 8, 32, 4, 0, 1, True, F32, 1.0, 1),     # more groups than it takes: one token to a wave
    (12300, 64, 16, 1, 1, 0, 0, True, F32, 1.0, 1),      # k too large for it
])
def test_route_score(L, T, E, k, G, keep, rank, sigmoid, bias, dt, scale, renorm):
    g = gen(T * 1000 + E)
    logits = normal(g, T, E, dtype=dt, scale=1.5)
    b = normal(g, E, scale=0.2) if bias else None
    ids, w = run_route(L, logits, k, bias=b, score=sigmoid, n_group=G, topk_group=keep, group_rank=rank, renorm=renorm,
                       scale=scale)
    want_ids, want_w = ref.route_score(f64(logits), k, sigmoid, None if b is None else f64(b), G, keep, rank == 1, renorm,
                                       scale)
    assert np.array_equal(ids, want_ids)
    # 64-bit arithmetic, one rounding to fp32
    close(w, want_w, U * (1 + 1e-6) * np.abs(want_w) + 1e-45, "weights")


@pytest.mark.parametrize("repeat", [1, 410, 1229])   # 10 rows, and enough for four tokens to a wave
def test_route_score_ties_and_specials(L, repeat):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(F32).min
    E = 70
    rows = torch.zeros(10, E)
    rows[1] = -inf                                    # nothing left
    rows[2] = nan
    rows[3] = -inf
    rows[3, 66] = 2.0                                 # one expert left
    rows[4, [3, 65]] = inf
    rows[5, ::2] = nan
    rows[6] = low
    rows[7, 5:60] = low
    rows[8] = torch.linspace(-90, 90, E)
    rows[9, 64:] = 1.0
    rows = rows.repeat(repeat, 1)
    for sigmoid in (0, 1):
        for G, keep, rank in ((1, 1, 0), (7, 2, 0), (7, 2, 1)):
            for bias in (None, torch.linspace(0.3, -0.3, E)):
                kw = dict(score=sigmoid, n_group=G, topk_group=keep, group_rank=rank)
                ids, w = run_route(L, rows.cuda(), 6, bias=None if bias is None else bias.cuda(), **kw)
                want_ids, want_w = ref.route_score(rows.double().numpy(), 6, sigmoid,
                                                   None if bias is None else bias.double().numpy(), G, keep, rank == 1)
                assert np.array_equal(ids, want_ids), (sigmoid, G, rank, bias is not None)
                close(w, want_w, U * (1 + 1e-6) * np.abs(want_w) + 1e-45, "weights")
                assert np.isfinite(w).all()
    # infinite and NaN biases: an excluded expert, a forced one, one that ranks last
    b = torch.zeros(E)
    b[0], b[1], b[2] = -inf, inf, nan
    ids, _ = run_route(L, torch.zeros(1, E).cuda(), 4, bias=b.cuda(), score=1)
    assert ids[0].tolist() == [1, 3, 4, 5]


@pytest.mark.parametrize("repeat", [1, 690])
def test_route_score_ties_and_specials_bf16(L, repeat):
    """16-bit logits without a bias: ties, signed zeros, masks, infinities and NaN."""
    inf, nan = float("inf"), float("nan")
    for E, G, keep in ((70, 1, 1), (70, 7, 2), (129, 1, 1), (256, 16, 1)):
        rows = torch.zeros(6, E)
        rows[1, ::2] = -0.0
        rows[2] = nan
        rows[2, E - 1] = -inf
        rows[3, 1::3] = inf
        rows[3, ::5] = nan
        rows[4] = torch.finfo(BF16).min
        rows[4, 5] = -inf
        rows[4, E - 2:] = torch.finfo(BF16).max
        rows[5] = (torch.arange(E) * 7 % 5).float() - 2
        l = rows.to(BF16).repeat(repeat, 1).cuda()
        for sigmoid in (0, 1):
            ids, w = run_route(L, l, 6, score=sigmoid, n_group=G, topk_group=keep)
            want_ids, want_w = ref.route_score(f64(l), 6, sigmoid, None, G, keep)
            assert np.array_equal(ids, want_ids), (E, G, sigmoid)
            close(w, want_w, U * (1 + 1e-6) * np.abs(want_w) + 1e-45, "weights")


@pytest.mark.parametrize("T", [40, 12289])
def test_route_score_saturated(L, T):
    """Without a bias the experts of the kept groups are ordered by their logits, also where the scores (and so the
    sums that rank the groups) are equal in 64 bits; equal logits go to the lower id."""
    g = gen(T)
    for logits, sigmoid in ((torch.randint(40, 60, (T, 96), generator=g, device="cuda").float(), 1),
                            (-1000.0 * torch.randint(1, 9, (T, 96), generator=g, device="cuda").float(), 0),
                            (normal(g, T, 96, dtype=BF16, scale=0.05).float(), 0)):
        for E, G, keep in ((96, 8, 3), (96, 48, 20), (64, 64, 20)):
            l = logits[:, :E]
            ids, w = run_route(L, l, 5, score=sigmoid, n_group=G, topk_group=keep, group_rank=1)
            want_ids, want_w = ref.route_score(f64(l), 5, sigmoid, None, G, keep, True)
            assert np.array_equal(ids, want_ids), (sigmoid, G)
            close(w, want_w, U * (1 + 1e-6) * np.abs(want_w) + 1e-45, "weights")


@pytest.mark.parametrize("T,E,k,G,keep,rank,sigmoid,bias,dt,scale,renorm", [
    (65, 340, 8, 1, 1, 0, 0, True, BF16, 2.5, 1), (7, 384, 20, 6, 2, 1, 1, True, F32, 1.0, 1),
    (13000, 260, 6, 26, 9, 1, 0, False, BF16, 1.0, 0), (33, 385, 5, 1, 1, 0, 0, True, F32, 1.0, 1),
    (11573, 60, 4, 4, 1, 1, 0, False, BF16, 1.0, 1), (18433, 256, 8, 8, 4, 1, 1, True, F32, 2.5, 1),
    (15362, 192, 12, 3, 2, 1, 0, True, BF16, 1.0, 1), (4101, 250, 15, 10, 2, 0, 1, False, BF16, 1.0, 0),
    (4096, 64, 6, 1, 1, 0, 0, False, BF16, 1.0, 1), (4097, 186, 9, 6, 4, 0, 0, False, BF16, 2.5, 1), (13831, 160, 6, 8, 3, 1, 0, False, F32, 1.0, 0),
])
def test_route_score_widths(L, T, E, k, G, keep, rank, sigmoid, bias, dt, scale, renorm):
    test_route_score(L, T, E, k, G, keep, rank, sigmoid, bias, dt, scale, renorm)


@pytest.mark.parametrize("sigmoid", [0, 1])
@pytest.mark.parametrize("T", [257, 12289])
def test_route_score_close_scores(L, sigmoid, T):
    """Scores whose differences with the bias lie below 32-bit rounding: the choice is the 64-bit one."""
    g = gen(77)
    E = 128
    for top2, G, keep in ((0, 1, 1), (0, 8, 3), (1, 8, 3)):
        base = normal(g, T, 1)
        logits = base + 2e-7 * torch.randint(-40, 41, (T, E), generator=g, device="cuda").float()
        b = (0.5 + 1e-8 * torch.randint(0, 16, (E,), generator=g, device="cuda").float())
        b[::9] -= 0.25
        ids, w = run_route(L, logits, 8, bias=b, score=sigmoid, n_group=G, topk_group=keep, group_rank=top2)
        want_ids, want_w = ref.route_score(f64(logits), 8, sigmoid, f64(b), G, keep, top2)
        # 64-bit scores that agree to 1e-15 may order either way between two programs
        same = ids == want_ids
        if not same.all():
            l = f64(logits)
            s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max(1, keepdims=True))
            s = s if sigmoid else s / s.sum(1, keepdims=True)
            c = s + f64(b)
            d = np.abs(np.take_along_axis(c, ids, 1) - np.take_along_axis(c, want_ids, 1))
            assert (d[~same] <= 1e-15).all(), (top2, G, d.max())
        assert same.mean() > 0.95


def test_route_score_strided_rows(L):
    g = gen(3)
    for dt in (F32, BF16):
        big = normal(g, 40, 131, dtype=dt)
        view = big[3:36:2, 1:130]
        assert view.stride(0) == 262
        ids, w = run_route(L, view, 5, score=1)
        want_ids, want_w = ref.route_score(f64(view), 5, 1)
        assert np.array_equal(ids, want_ids)
        close(w, want_w, U * (1 + 1e-6) * np.abs(want_w), "weights")


def test_route_score_equals_route_topk_without_bias(L):
    """Softmax, no bias, no groups: the choice and weights of route_topk on the same logits."""
    g = gen(5)
    logits = normal(g, 300, 128)
    ids, w = run_route(L, logits, 8)
    i0 = torch.empty(300, 8, dtype=torch.int32, device="cuda")
    w0 = torch.empty(300, 8, device="cuda")
    L.route_topk(logits, 8, i0, w0)
    assert np.array_equal(ids, i0.cpu().numpy())
    assert np.abs(w - f64(w0)).max() <= 1e-5      # the bound of route_topk's own weights


# --------------------------------------------------------------- norms ----
NORM_CASES = [
    (1, 8, F32, F32, 0.0), (1, 2816, BF16, BF16, 1.0), (3, 64, BF16, F32, 0.0), (16, 2816, BF16, BF16, 0.0),
    (5, 520, F32, BF16, 1.0), (2, 8200, F32, BF16, 0.0), (2, 16392, BF16, BF16, 1.0), (2, 32768, F32, F32, 0.0),
    (2050, 136, BF16, BF16, 0.0), (2049, 2824, F32, BF16, 1.0), (2048, 4104, F32, F32, 0.0),
]


@pytest.mark.parametrize("T,H,ht,xt,off", NORM_CASES)
def test_norm_in(L, T, H, ht, xt, off):
    g = gen(T + H)
    wt = BF16 if H % 3 else F32
    h, hbuf = padded(T, H, ht, 16, 3.0)
    h.copy_(normal(g, T, H) * (0.1 + 10 * torch.rand(T, 1, generator=g, device="cuda")))
    w = normal(g, H, dtype=wt, scale=0.3) + (1 - off)
    w = w.to(wt)
    x, xbuf = padded(T, H, xt, 8, 5.0)
    q, qbuf = padded(T, H, torch.int8, 24, 77)
    sc = torch.full((T + 1,), 9.0, device="cuda")
    L.norm_in(h, w, EPS, x=x, xq=q, xq_scale=sc[:T], w_offset=off)
    x2 = torch.empty(T, H, dtype=xt, device="cuda")
    L.norm_in(h, w, EPS, x=x2, w_offset=off)
    torch.cuda.synchronize()
    check_padding(xbuf, H, 5.0)
    check_padding(qbuf, H, 77)
    assert sc[T] == 9.0
    assert torch.equal(x, x2), "x depends on whether codes are written too"
    want, r = ref.norm_in(f64(h), f64(w), off, EPS)
    close(f64(x), want, np.abs(want) * (ref.NORM_U + half_step(xt) * (1 + ref.NORM_U)) + 1e-37, "x")
    qw, s = ref.codes(ref.unnormed(h.float().cpu().numpy(), w.float().cpu().numpy(), off))
    assert np.array_equal(q.cpu().numpy(), qw), "codes differ"
    close(f64(sc[:T]), s * r[:, 0], s * r[:, 0] * ref.NORM_U + 1e-37, "scales")


def test_norm_in_without_weight_and_specials(L):
    inf, nan = float("inf"), float("nan")
    h = torch.randn(7, 64, generator=torch.Generator().manual_seed(1))
    h[1] = 0
    h[2, 5] = nan
    h[3, 60] = inf
    h[4, 0] = -inf
    h[5] = 1e-30
    h[6] = 1e15
    h = h.cuda()
    x = torch.empty_like(h)
    q = torch.empty(7, 64, dtype=torch.int8, device="cuda")
    sc = torch.empty(7, device="cuda")
    L.norm_in(h, None, EPS, x=x, xq=q, xq_scale=sc)
    torch.cuda.synchronize()
    ok = [0, 1, 5, 6]
    want, r = ref.norm_in(f64(h)[ok], None, 0, EPS)
    close(f64(x)[ok], want, np.abs(want) * (ref.NORM_U + U) + 1e-37, "x")
    qw, s = ref.codes(h.cpu().numpy()[ok])
    assert np.array_equal(q.cpu().numpy()[ok], qw)
    close(f64(sc)[ok], s * r[:, 0], s * r[:, 0] * ref.NORM_U + 1e-37, "scales")
    assert (x[1] == 0).all() and (q[1] == 0).all() and sc[1] == 0
    assert torch.isnan(x[2]).all() and not torch.isfinite(sc[2])
    assert not torch.isfinite(sc[3]) and not torch.isfinite(sc[4])
    assert torch.isnan(x[3, 60]) and torch.isnan(x[4, 0])


@pytest.mark.parametrize("T,K,xt", [(1, 16, F32), (16, 704, BF16), (3, 2112, F32), (2049, 704, BF16), (2, 32768, BF16),
                                    (70, 8, BF16)])
def test_quantize_tokens(L, T, K, xt):
    g = gen(K)
    x, _ = padded(T, K, xt, 8, 1.0)
    x.copy_(normal(g, T, K))
    if T > 2:
        x[1] = 0
    q, qbuf = padded(T, K, torch.int8, 8, 55)
    sc = torch.empty(T, device="cuda")
    L.quantize_tokens(x, q, sc)
    torch.cuda.synchronize()
    check_padding(qbuf, K, 55)
    qw, s = ref.codes(x.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), qw) and np.array_equal(sc.cpu().numpy(), s)
    if xt == BF16 and T <= 16:   # the weight quantiser's rule but for the rounding of the step
        xc = x.contiguous()
        q2 = torch.empty(T, K, dtype=torch.int8, device="cuda")
        s2 = torch.empty(T, device="cuda")
        L.quantize(L.W_INT8_ROW, xc.view(torch.int16), q2, s2)
        close(f64(sc), f64(s2), 2 * U * f64(s2), "step")
        assert (q2.int() - q.int()).abs().max() <= 1


@pytest.mark.parametrize("T,H,k,rt,yt,ht,gate,off,drop,nxt", [
    (1, 8, 1, F32, None, F32, None, 0.0, 0.0, "x"),
    (1, 2816, 8, F32, BF16, BF16, "channel", 1.0, 0.0, "xq"),
    (16, 2816, 8, F32, BF16, BF16, "token", 0.0, 0.2, "both"),
    (7, 520, 3, BF16, F32, F32, "full", 1.0, 0.9, "both"),
    (4, 16392, 10, BF16, None, BF16, "channel", 0.0, 0.1, "x"),
    (3, 32768, 9, F32, F32, F32, None, 1.0, 0.1, "xq"),
    (5, 1024, 32, F32, None, BF16, None, 0.0, 0.5, None),
    (6, 64, 0, F32, BF16, F32, "token", 0.0, 0.0, "x"),
    (1100, 264, 6, BF16, BF16, BF16, "channel", 0.0, 0.1, "both"),
    (9, 704, 8, F32, None, BF16, "channel", 0.0, 1.0, "x"),     # every route dropped
])
def test_norm_out(L, T, H, k, rt, yt, ht, gate, off, drop, nxt):
    g = gen(T * 31 + H + k)
    R = T * k
    h, _ = padded(T, H, ht, 8, 1.0)
    h.copy_(normal(g, T, H, scale=3.0))
    routes = normal(g, R, H, dtype=rt) if k else None
    pos = tw = None
    if k:
        pos = torch.randperm(R, generator=g, device="cuda").to(torch.int32).view(T, k)
        gone = torch.rand(T, k, generator=g, device="cuda") < drop
        used = pos.clone()
        pos = torch.where(gone, torch.full_like(pos, -1), pos)
        routes[used[gone].long()] = float("nan")        # a dropped route's row is never read as a number
        tw = torch.rand(T, k, generator=g, device="cuda")
    y = None
    if yt is not None:
        y, _ = padded(T, H, yt, 8, 1.0)
        y.copy_(normal(g, T, H))
    gt = None
    if gate is not None:
        shape = {"channel": (1, H), "token": (T, 1), "full": (T, H)}[gate]
        gt = normal(g, *shape, dtype=BF16 if gate == "full" else F32)
    wp = (normal(g, H, scale=0.2) + (1 - off)).to(BF16)
    wn = (normal(g, H, scale=0.2) + (1 - off)).to(BF16)
    ho, hbuf = padded(T, H, ht, 16, 4.0)
    kw = {}
    if nxt in ("x", "both"):
        kw["x"], xbuf = padded(T, H, BF16, 8, 6.0)
    if nxt in ("xq", "both"):
        kw["xq"], qbuf = padded(T, H, torch.int8, 16, 33)
        kw["xq_scale"] = torch.empty(T, device="cuda")
    if nxt:
        kw["w_next"] = wn
    L.norm_out(h, ho, wp, EPS, out_routes=routes, topk_w=tw, route_pos=pos, y=y, gate=gt, block_scale=0.7, res_scale=1.3,
               w_offset=off, **kw)
    torch.cuda.synchronize()
    check_padding(hbuf, H, 4.0)
    want, bound = ref.norm_out(f64(h), None if routes is None else np.nan_to_num(f64(routes)),
                               None if tw is None else f64(tw), None if pos is None else pos.cpu().numpy(),
                               None if y is None else f64(y), f64(wp), off, EPS, None if gt is None else f64(gt),
                               np.float64(np.float32(0.7)), np.float64(np.float32(1.3)))
    close(f64(ho), want, bound + half_step(ht) * (np.abs(want) + bound), "h_out")
    # the next norm is that of the rows as stored: the codes are those of the norm of them alone
    if nxt:
        x2 = torch.empty(T, H, dtype=BF16, device="cuda")
        q2 = torch.empty(T, H, dtype=torch.int8, device="cuda")
        s2 = torch.empty(T, device="cuda")
        L.norm_in(ho, wn, EPS, x=x2, xq=q2, xq_scale=s2, w_offset=off)
        want_x, r = ref.norm_in(f64(ho), f64(wn), off, EPS)
        if "x" in kw:
            check_padding(xbuf, H, 6.0)
            close(f64(kw["x"]), want_x, np.abs(want_x) * (ref.NORM_U + half_step(BF16) * (1 + ref.NORM_U)) + 1e-37, "x")
        if "xq" in kw:
            check_padding(qbuf, H, 33)
            assert torch.equal(kw["xq"].contiguous(), q2)
            close(f64(kw["xq_scale"]), f64(s2), 2 * ref.NORM_U * f64(s2) + 1e-37, "scales")
    # in place
    h2 = h.clone()
    L.norm_out(h2, h2, wp, EPS, out_routes=routes, topk_w=tw, route_pos=pos, y=y, gate=gt, block_scale=0.7, res_scale=1.3,
               w_offset=off)
    assert torch.equal(h2, ho), "in place differs"


def test_norm_out_without_post_norm_is_the_combine(L):
    """w_post None, no gate, residual 0: b itself, which is combine's y."""
    g = gen(9)
    T, H, k = 33, 704, 6
    routes = normal(g, T * k, H)
    pos = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    pos[3] = -1
    pos[5, 2] = T * k + 5          # outside: dropped, not read
    tw = torch.rand(T, k, generator=g, device="cuda")
    y0 = torch.empty(T, H, device="cuda")
    pos_in = torch.where(pos >= T * k, torch.full_like(pos, -1), pos)
    L.combine(routes, tw, pos_in, y0)
    h = torch.zeros(T, H, device="cuda")
    ho = torch.empty_like(h)
    L.norm_out(h, ho, None, EPS, out_routes=routes, topk_w=tw, route_pos=pos, res_scale=0.0)
    close(f64(ho), f64(y0), 16 * U * np.abs(f64(routes)).max() * k, "combine")


# rows that share a workgroup, with a ragged last one: 16, 32 and 64 lanes
@pytest.mark.parametrize("T,H,ht,xt,off", [(17, 8, F32, BF16, 1.0), (4099, 128, BF16, BF16, 1.0), (31, 136, F32, F32, 0.0),
                                           (2057, 256, BF16, F32, 0.0), (3, 264, F32, BF16, 1.0), (1029, 512, BF16, BF16, 0.0)])
def test_norm_in_short_rows(L, T, H, ht, xt, off):
    test_norm_in(L, T, H, ht, xt, off)


@pytest.mark.parametrize("T,K,xt", [(15, 128, F32), (4097, 64, BF16), (9, 256, BF16), (33, 248, F32), (6, 512, BF16)])
def test_quantize_short_rows(L, T, K, xt):
    test_quantize_tokens(L, T, K, xt)


@pytest.mark.parametrize("T,H,k,rt,yt,ht,gate,off,drop,nxt", [
    (1, 512, 8, F32, BF16, BF16, "channel", 1.0, 0.0, "both"), (5, 504, 5, BF16, None, F32, "token", 0.0, 0.3, "xq"),
    (2051, 64, 4, F32, BF16, BF16, "full", 1.0, 0.1, "both"), (7, 128, 32, BF16, F32, F32, None, 0.0, 0.5, "x"),
])
def test_norm_out_short_rows(L, T, H, k, rt, yt, ht, gate, off, drop, nxt):
    test_norm_out(L, T, H, k, rt, yt, ht, gate, off, drop, nxt)


# ------------------------------------------------------------ products ----
def rand_codes(g, rows, K, pad=0, extreme=False):
    buf = torch.randint(-127, 128, (rows, K + pad), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    if extreme:
        buf.fill_(-128)
    return buf[:, :K]


MM_CASES = [
    # T, N, K, out, bias
    (1, 1, 16, F32, False), (1, 5632, 2816, BF16, False), (2, 17, 32, BF16, True), (15, 704, 2816, F32, True),
    (16, 33, 704, BF16, False), (17, 100, 1424, F32, False), (31, 2816, 704, BF16, True), (33, 65, 48, F32, True),
    (64, 130, 4096, BF16, False), (65, 129, 144, F32, True), (77, 2819, 1424, F32, False), (128, 256, 128, BF16, True),
    (129, 257, 272, BF16, False), (200, 1000, 2816, F32, True), (300, 50, 8192, F32, False), (1024, 1408, 704, BF16, False),
    (1000, 4099, 400, BF16, True), (3000, 4500, 144, F32, True), (2560, 5200, 256, BF16, False), (9, 64, 131056, F32, False),
]


@pytest.mark.parametrize("T,N,K,ot,bias", MM_CASES)
def test_matmul_i8(L, T, N, K, ot, bias):
    print(f"[case] matmul_i8 T={T} N={N} K={K} {ot} bias={bias}", flush=True)
    g = gen(T + N + K)
    xq, wq = rand_codes(g, T, K, 16), rand_codes(g, N, K, 32)
    sx = torch.rand(T, generator=g, device="cuda") * 0.01
    sw = torch.rand(N, generator=g, device="cuda") * 0.01
    b = normal(g, N) if bias else None
    out, buf = padded(T, N, ot, 5 if N % 2 else 8, 2.0)
    L.matmul_i8(xq, sx, wq, sw, out, bias=b)
    torch.cuda.synchronize()
    check_padding(buf, N, 2.0)
    want, bound = ref.matmul_i8(xq.cpu().numpy(), f64(sx), wq.cpu().numpy(), f64(sw), None if b is None else f64(b))
    close(f64(out), want, bound + half_step(ot) * (np.abs(want) + bound), "out")


def test_matmul_i8_largest_sums(L):
    """Every product 128 * 128 at the largest K: sums just below 2^31, exact in every path."""
    K = 131056
    for T, N in ((3, 20), (70, 70)):
        g = gen(1)
        xq, wq = rand_codes(g, T, K, extreme=True), rand_codes(g, N, K, extreme=True)
        out = torch.empty(T, N, device="cuda")
        L.matmul_i8(xq, torch.ones(T, device="cuda"), wq, torch.ones(N, device="cuda"), out)
        assert (out == float(np.float32(128 * 128 * K))).all()


@pytest.mark.parametrize("T,F,K,ot,act", [
    (1, 2112, 2816, BF16, 0), (1, 1, 16, F32, 1), (16, 704, 2816, F32, 1), (16, 2112, 2816, BF16, 0), (30, 100, 704, BF16, 1),
    (63, 65, 400, F32, 0), (77, 63, 1424, F32, 0), (130, 129, 144, BF16, 1), (1024, 704, 256, BF16, 0),
    (600, 10000, 64, F32, 1), (2300, 3001, 208, BF16, 0),
])
def test_gated_matmul_i8(L, T, F, K, ot, act):
    print(f"[case] gated_matmul_i8 T={T} F={F} K={K} {ot} act={act}", flush=True)
    g = gen(T + F + K)
    xq, wq = rand_codes(g, T, K, 16), rand_codes(g, 2 * F, K, 16)
    # products of order 1 to 10, some gates far out
    s = 3.0 / (73.0 * 73.0 * K ** 0.5)
    sx = (0.2 + torch.rand(T, generator=g, device="cuda")) * s
    sw = 0.2 + torch.rand(2 * F, generator=g, device="cuda") * (1.0 if F < 500 else 4.0)
    out, buf = padded(T, F, ot, 3, 2.0)
    L.gated_matmul_i8(xq, sx, wq, sw, act, out)
    torch.cuda.synchronize()
    check_padding(buf, F, 2.0)
    v, _ = ref.matmul_i8(xq.cpu().numpy(), f64(sx), wq.cpu().numpy(), f64(sw))
    want, bound = ref.gated(v[:, :F], v[:, F:], act)
    close(f64(out), want, bound + half_step(ot) * (np.abs(want) + bound), "out")


# one shape per tile, ragged on every side
@pytest.mark.parametrize("T,N,K,ot,bias", [
    (50, 130, 1424, F32, True), (130, 2053, 1424, BF16, True), (77, 4101, 2816, F32, False), (77, 130, 400, BF16, True),
    (200, 4101, 272, F32, True), (200, 8200, 272, BF16, True), (1030, 4101, 272, F32, True), (1030, 4101, 272, BF16, False),
    (3000, 2053, 400, F32, False), (1030, 8200, 272, BF16, True), (200, 4101, 2816, BF16, False), (1030, 8200, 400, F32, True),
    (2100, 4101, 400, BF16, True),
    # rows that can be stored in 16-byte pieces
    (77, 128, 400, F32, False), (200, 4104, 2816, BF16, True), (1030, 4104, 272, BF16, False), (3000, 2056, 400, F32, True),
    (33, 2056, 400, BF16, True), (48, 4096, 272, F32, False), (64, 2000, 2816, BF16, False), (64, 2000, 2832, BF16, True),
    (49, 77, 144, F32, True),
])
def test_matmul_i8_tiles(L, T, N, K, ot, bias):
    test_matmul_i8(L, T, N, K, ot, bias)


@pytest.mark.parametrize("T,F,K,ot,act", [
    (77, 130, 1424, BF16, 0), (200, 601, 1424, F32, 1), (200, 1100, 2816, BF16, 1), (77, 130, 272, F32, 0),
    (77, 4101, 272, BF16, 0), (200, 4101, 272, F32, 0), (1030, 2053, 272, BF16, 0), (1030, 2053, 272, F32, 1),
    (3000, 1100, 400, BF16, 1), (1030, 4101, 272, F32, 0), (77, 4101, 2816, F32, 1), (1030, 4101, 400, BF16, 0),
    (2100, 2053, 400, F32, 1), (1030, 2056, 272, BF16, 1), (77, 4104, 2816, BF16, 0), (3000, 1104, 400, F32, 0),
    (40, 1000, 704, BF16, 0), (64, 2048, 1424, F32, 1), (33, 5, 16, BF16, 1),
])
def test_gated_matmul_i8_tiles(L, T, F, K, ot, act):
    test_gated_matmul_i8(L, T, F, K, ot, act)


# either side of the token and row counts where few tokens go over to tiles
@pytest.mark.parametrize("T,N,K,ot,bias", [
    (1, 15, 16, BF16, True), (2, 4099, 144, F32, True), (16, 8192, 4096, BF16, False), (16, 16, 112, F32, False),
    (17, 4096, 400, BF16, True), (17, 4097, 400, BF16, True), (18, 48, 131056, F32, False), (32, 1000, 1424, F32, True),
    (32, 4200, 704, BF16, False), (33, 1000, 1424, F32, True),
])
def test_matmul_i8_few_tokens(L, T, N, K, ot, bias):
    test_matmul_i8(L, T, N, K, ot, bias)


@pytest.mark.parametrize("T,F,K,ot,act", [
    (1, 7, 16, F32, 0), (5, 2049, 528, BF16, 1), (16, 9, 1424, BF16, 0), (17, 2048, 400, F32, 0), (17, 2049, 400, F32, 1),
    (32, 300, 2816, BF16, 0), (32, 2100, 272, BF16, 1),
])
def test_gated_matmul_i8_few_tokens(L, T, F, K, ot, act):
    test_gated_matmul_i8(L, T, F, K, ot, act)


def test_matmul_i8_non_finite_scales(L):
    """A token whose scale is NaN or infinite gives NaN there and leaves the others alone."""
    g = gen(2)
    for T in (4, 100):
        xq, wq = rand_codes(g, T, 64), rand_codes(g, 40, 64)
        xq[1] = 0
        sx = torch.ones(T, device="cuda")
        sx[1], sx[2] = float("inf"), float("nan")
        out = torch.empty(T, 40, device="cuda")
        L.matmul_i8(xq, sx, wq, torch.ones(40, device="cuda"), out)
        assert torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
        keep = [0] + list(range(3, T))
        want, bound = ref.matmul_i8(xq.cpu().numpy()[keep], np.ones(len(keep)), wq.cpu().numpy(), np.ones(40))
        close(f64(out)[keep], want, bound, "out")


def test_binding_refusals_on_gpu_tensors(L):
    """Wrong shapes, types and layouts are refused before anything is enqueued."""
    z = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")
    i8, i32 = torch.int8, torch.int32
    h, x, w = z(4, 64, dt=BF16), z(4, 64, dt=BF16), z(64)
    ids, tw = z(4, 2, dt=i32), z(4, 2)
    for err, call in [
        (ValueError, lambda: L.route_score_topk(z(8), 2, ids, tw)),
        (ValueError, lambda: L.route_score_topk(z(4, 8), 3, ids, tw)),
        (TypeError, lambda: L.route_score_topk(z(4, 8, dt=torch.float16), 2, ids, tw)),
        (TypeError, lambda: L.route_score_topk(z(4, 8), 2, ids.long(), tw)),
        (ValueError, lambda: L.route_score_topk(z(8, 4).t(), 2, ids, tw)),
        (ValueError, lambda: L.route_score_topk(z(4, 8), 2, ids, tw, bias=z(9))),
        (ValueError, lambda: L.route_score_topk(z(4, 8), 2, ids, tw, bias=torch.zeros(8))),
        (L.MoeError, lambda: L.route_score_topk(z(4, 8), 2, ids, tw, n_group=3)),
        (ValueError, lambda: L.norm_in(h, z(65), EPS, x=x)),
        (ValueError, lambda: L.norm_in(h, w, EPS, x=z(4, 72, dt=BF16))),
        (ValueError, lambda: L.norm_in(h, w, EPS, xq=z(4, 64, dt=i8))),
        (TypeError, lambda: L.norm_in(h, w, EPS, xq=z(4, 64, dt=torch.uint8), xq_scale=z(4))),
        (L.MoeError, lambda: L.norm_in(h, w, EPS)),
        (L.MoeError, lambda: L.norm_in(h, w, 0.0, x=x)),
        (L.MoeError, lambda: L.norm_in(h, w, EPS, x=h)),
        (L.MoeError, lambda: L.norm_in(z(4, 60), None, EPS, x=z(4, 60))),
        (L.MoeError, lambda: L.norm_in(z(4, 66)[:, 1:65], None, EPS, x=x)),
        (L.MoeError, lambda: L.norm_in(z(1, 64).expand(4, 64), None, EPS, x=x)),
        (TypeError, lambda: L.norm_out(h, z(4, 64), None, EPS, y=x)),
        (ValueError, lambda: L.norm_out(h, x, None, EPS, y=z(3, 64))),
        (ValueError, lambda: L.norm_out(h, x, None, EPS, out_routes=z(8, 64))),
        (ValueError, lambda: L.norm_out(h, x, None, EPS, out_routes=z(8, 64), topk_w=z(4, 2), route_pos=z(7, dt=i32))),
        (ValueError, lambda: L.norm_out(h, x, None, EPS, y=z(4, 64), gate=z(3, 64))),
        (ValueError, lambda: L.norm_out(h, x, None, EPS, y=z(4, 64), gate=z(2, 4, 64))),
        (ValueError, lambda: L.norm_out(h, x, None, EPS, y=z(4, 64), w_next=w)),
        (TypeError, lambda: L.norm_out(h, x, w, EPS, y=z(4, 64), w_next=w.bfloat16(), x=z(4, 64))),
        (L.MoeError, lambda: L.norm_out(h, x, None, EPS)),
        (L.MoeError, lambda: L.norm_out(h, x, None, EPS, y=z(4, 64), gate=z(64, 4).t())),
        (ValueError, lambda: L.matmul_i8(z(4, 64, dt=i8), z(4), z(8, 48, dt=i8), z(8), z(4, 8))),
        (ValueError, lambda: L.matmul_i8(z(4, 64, dt=i8), z(3), z(8, 64, dt=i8), z(8), z(4, 8))),
        (TypeError, lambda: L.matmul_i8(z(4, 64), z(4), z(8, 64, dt=i8), z(8), z(4, 8))),
        (TypeError, lambda: L.matmul_i8(z(4, 64, dt=i8), z(4), z(8, 64, dt=i8), z(8), z(4, 8, dt=torch.float16))),
        (L.MoeError, lambda: L.matmul_i8(z(4, 72, dt=i8), z(4), z(8, 72, dt=i8), z(8), z(4, 8))),
        (ValueError, lambda: L.gated_matmul_i8(z(4, 64, dt=i8), z(4), z(7, 64, dt=i8), z(7), 0, z(4, 3))),
        (L.MoeError, lambda: L.gated_matmul_i8(z(4, 64, dt=i8), z(4), z(8, 64, dt=i8), z(8), 9, z(4, 4))),
    ]:
        with pytest.raises(err):
            call()


def test_empty_batches(L):
    """T = 0: nothing is written, nothing refused."""
    z = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")
    i8 = torch.int8
    L.route_score_topk(z(0, 8), 2, z(0, 2, dt=torch.int32), z(0, 2))
    L.norm_in(z(0, 64), z(64), EPS, x=z(0, 64), xq=z(0, 64, dt=i8), xq_scale=z(0))
    L.norm_out(z(0, 64), z(0, 64), z(64), EPS, y=z(0, 64))
    L.quantize_tokens(z(0, 64), z(0, 64, dt=i8), z(0))
    L.matmul_i8(z(0, 64, dt=i8), z(0), z(8, 64, dt=i8), z(8), z(0, 8))
    L.gated_matmul_i8(z(0, 64, dt=i8), z(0), z(8, 64, dt=i8), z(8), 0, z(0, 4))
    torch.cuda.synchronize()


@pytest.mark.parametrize("shape", [(64,), (1, 64), (5, 1), (5, 64), (1,), (1, 1), ()])
def test_norm_out_gate_broadcasts(L, shape):
    g = gen(4)
    h, y = normal(g, 5, 64), normal(g, 5, 64)
    gate = normal(g, *shape) if shape else normal(g, 1).reshape(())
    a, b = torch.empty_like(h), torch.empty_like(h)
    L.norm_out(h, a, None, EPS, y=y, gate=gate)
    L.norm_out(h, b, None, EPS, y=y, gate=gate.expand(5, 64).contiguous())
    assert torch.equal(a, b)
    close(f64(a), f64(h) + f64(y) * f64(gate), 3 * U * (np.abs(f64(h)) + np.abs(f64(y) * f64(gate))) + 1e-37, "h_out")

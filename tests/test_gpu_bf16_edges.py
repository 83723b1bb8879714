"""The bfloat16 products where they can go wrong: every tile with its ring run around, adapters that hold infinities
and NaN, rows and pools whose offsets pass 32 bits, far gates, replayed graphs, several streams, repeated runs."""
import numpy as np
import pytest
import torch

import bf16_cases as bc
import bf16_ref as ref
import block_ref
from bf16_ref import BF16, F32, F64, whole
from block_ref import f64, half_step
from test_gpu_bf16 import equal, make_adapters, strided
from test_gpu_block import L, check_padding, close, gen, normal, padded  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu


def by_tile(shapes):
    return [pytest.param(*s, id=f"tile{i}-" + "x".join(map(str, s))) for i, s in sorted(shapes.items())]


@pytest.mark.parametrize("T,N,K", by_tile(bc.shapes("MAT_NT")))
def test_every_tile(L, T, N, K):  # noqa: F811
    g = gen(T + N + K)
    x, w = whole(g, T, K), whole(g, N, K, top=3)
    for dt, pad in ((F32, 8 + -N % 8), (BF16, 3)):
        out, buf = padded(T, N, dt, pad, 2.0)
        L.matmul_bf16(x, w, out)
        torch.cuda.synchronize()
        check_padding(buf, N, 2.0)
        equal(out, x.to(F64) @ w.to(F64).t().contiguous(), "out")


@pytest.mark.parametrize("T,F,K", by_tile(bc.shapes("MAT_GATED")))
def test_every_gated_tile(L, T, F, K):  # noqa: F811
    g = gen(T + F + K)
    x, w = whole(g, T, K), whole(g, 2 * F, K, unit=2.0 ** -6)
    v = x.to(F64) @ w.to(F64).t().contiguous()
    want, bound = block_ref.gated(v[:, :F].cpu().numpy(), v[:, F:].cpu().numpy(), 0)
    for dt in (F32, BF16):
        out, buf = padded(T, F, dt, 3 if F % 2 else 8, 2.0)
        pre, pbuf = padded(T, 2 * F, BF16, 8 + -2 * F % 8, 2.0)
        L.gated_matmul_bf16(x, w, 0, out, pre=pre)
        torch.cuda.synchronize()
        check_padding(buf, F, 2.0)
        check_padding(pbuf, 2 * F, 2.0)
        equal(pre, v, "pre")
        close(f64(out), want, bound + half_step(dt) * (abs(want) + bound), "out")


@pytest.mark.parametrize("rows,cols,k", by_tile(bc.shapes("MAT_NN")))
def test_every_tile_of_the_rows_gradient(L, rows, cols, k):  # noqa: F811
    g = gen(rows + cols + k)
    d, w = whole(g, rows, k), whole(g, k, cols)
    dx, buf = padded(rows, cols, BF16, 8, 2.0)
    L.matmul_bf16_backward(torch.empty(rows, cols, dtype=BF16, device="cuda"), w, d, dx=dx)
    torch.cuda.synchronize()
    check_padding(buf, cols, 2.0)
    equal(dx, d.to(F64) @ w.to(F64), "dx")


@pytest.mark.parametrize("rows,cols,k", by_tile(bc.shapes("MAT_TN")))
def test_every_tile_of_the_weights_gradient(L, rows, cols, k):  # noqa: F811
    g = gen(rows + cols + k)
    d, x = whole(g, k, rows), whole(g, k, cols)
    dw, buf = padded(rows, cols, F32, 3, 2.0)
    L.matmul_bf16_backward(x, torch.empty(rows, cols, dtype=BF16, device="cuda"), d, dw=dw)
    torch.cuda.synchronize()
    check_padding(buf, cols, 2.0)
    equal(dw, d.to(F64).t().contiguous() @ x.to(F64), "dw")


@pytest.mark.parametrize("T,N,K", by_tile(bc.pair_shapes()))
def test_every_pair(L, T, N, K):  # noqa: F811
    g = gen(T + N + K)
    x, w, d = strided(whole(g, T, K)), strided(whole(g, N, K)), strided(whole(g, T, N))
    dx, xbuf = padded(T, K, F32, 8, 2.0)
    dw, wbuf = padded(N, K, BF16, 1, 2.0)
    L.matmul_bf16_backward(x, w, d, dx=dx, dw=dw)
    torch.cuda.synchronize()
    check_padding(xbuf, K, 2.0)
    check_padding(wbuf, K, 2.0)
    equal(dx, d.to(F64) @ w.to(F64).contiguous(), "dx")
    equal(dw, d.to(F64).t().contiguous() @ x.to(F64).contiguous(), "dw")


@pytest.mark.parametrize("gated,kind", [(False, "tokens"), (True, "tokens"), (False, "runs"), (True, "runs")])
@pytest.mark.parametrize("R", [16, 72])
def test_every_tile_with_adapters(L, gated, kind, R):  # noqa: F811
    for T, N, K in bc.shapes("MAT_GATED" if gated else "MAT_NT", True).values():
        print(f"[case] adapters gated={gated} {kind} R={R} T={T} N={N} K={K}", flush=True)
        g, halves, n = gen(T + N + K + R), 2 if gated else 1, 11
        x, w, a, b, ids, scale = make_adapters(g, T, K, N, n, R, halves, kind)
        ranks = torch.randint(0, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
        low, up = ref.adapters(x, ids, a, b, scale, ranks, halves)
        s = torch.empty(T, halves * R, dtype=BF16, device="cuda")
        L.adapter_shrink(x, ids, a if gated else a[:, 0], scale, s, ranks=ranks)
        equal(s, low, "s")
        v = x.to(F64) @ w.to(F64).t().contiguous() + up
        out = torch.empty(T, N, dtype=F32, device="cuda")
        if gated:
            pre = torch.empty(T, 2 * N, dtype=BF16, device="cuda")
            L.gated_matmul_bf16(x, w, 0, out, pre=pre, s=s, adapter_ids=ids, b=b, ranks=ranks)
            equal(pre, v, "pre")
        else:
            L.matmul_bf16(x, w, out, s=s, adapter_ids=ids, b=b, ranks=ranks)
            equal(out, v, "out")


@pytest.mark.parametrize("T", [1, 16, 40, 61, 129, 700, 3001])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("R", [16, 64])
def test_a_broken_adapter_stays_with_its_tokens(L, T, gated, R):  # noqa: F811
    """Infinities and NaN of one adapter, or of one token's row, reach no other request's row."""
    n, N, K, halves = 5, 328, 264, 2 if gated else 1
    g = gen(T + R)
    x, w, a, b, _, scale = make_adapters(g, T, K, N, n, R, halves, "tokens")
    ids = (torch.arange(T, device="cuda") % n).to(torch.int32)
    clean = torch.empty(T, N, device="cuda")
    run = lambda xx, aa, bb, out: (
        s.fill_(9.0), L.adapter_shrink(xx, ids, aa if gated else aa[:, 0], scale, s),
        L.gated_matmul_bf16(xx, w, 1, out, s=s, adapter_ids=ids, b=bb) if gated else L.matmul_bf16(xx, w, out, s=s, adapter_ids=ids, b=bb))
    s = torch.empty(T, halves * R, dtype=BF16, device="cuda")
    run(x, a, b, clean)
    assert torch.isfinite(clean).all()
    for what in ("a", "b", "x"):
        x2, a2, b2 = x.clone(), a.clone(), b.clone()
        if what == "a":
            a2[2, :, 3, 7] = float("inf")
            a2[2, :, 5] = float("nan")
            hit = ids == 2
        elif what == "b":
            b2[2, 1::2, 1] = float("nan")
            b2[2, ::3, R - 1] = float("inf")
            hit = ids == 2
        else:
            x2[T // 2, 5] = float("nan")
            hit = torch.arange(T, device="cuda") == T // 2
        out = torch.empty_like(clean)
        run(x2, a2, b2, out)
        assert torch.equal(out[~hit], clean[~hit]), what
        if hit.any():
            assert not torch.isfinite(out[hit]).all(), what


def test_far_rows_and_pools(L):  # noqa: F811
    """Rows and adapters whose element offsets pass 2^32."""
    T, N, K, R, far = 4200, 136, 72, 16, 1 << 20
    g = gen(3)
    big = torch.empty(T * far + 4096, dtype=BF16, device="cuda")          # 8.8 GB
    assert T * far > 1 << 32
    x = big[:T * far].view(T, far)[:, :K]
    x.copy_(whole(g, T, K, top=1))
    s = torch.empty(T * far, dtype=BF16, device="cuda").view(T, far)[:, :R]   # (an output is refused between an input's rows)
    d = big[2048:2048 + T * far].view(T, far)[:, :N]
    d.copy_(whole(g, T, N))
    w = whole(g, N, K)
    n, stride = 3, (1 << 31) + 64
    pool = torch.empty(2 * stride + 65536, dtype=BF16, device="cuda")     # 8.6 GB
    a = torch.as_strided(pool, (n, R, K), (stride, K, 1))
    b = torch.as_strided(pool, (n, N, R), (stride, R, 1), 8192)
    a.copy_(whole(g, n, R, K, top=1))
    b.copy_(whole(g, n, N, R))
    ids = torch.randint(0, n, (T,), generator=g, device="cuda").to(torch.int32)
    L.adapter_shrink(x, ids, a, None, s)
    low, up = ref.adapters(x.contiguous(), ids, a.contiguous()[:, None], b.contiguous(), None, None, 1)
    equal(s, low, "s")
    fbuf = torch.empty(T * far, device="cuda")                            # 17.6 GB
    out = fbuf.view(T, far)[:, 8:8 + N]
    L.matmul_bf16(x, w, out, s=s, adapter_ids=ids, b=b)
    v = x.to(F64) @ w.to(F64).t().contiguous() + up
    equal(out, v, "out")
    dx, dw = fbuf.view(T, far)[:, 512:512 + K], torch.empty(N, K, device="cuda")
    L.matmul_bf16_backward(x, w, d, dx=dx, dw=dw)
    equal(dx, d.to(F64) @ w.to(F64), "dx")
    equal(dw, d.to(F64).t().contiguous() @ x.to(F64), "dw")


@pytest.mark.parametrize("act", [0, 1])
def test_far_gates(L, act):  # noqa: F811
    """The activation's gradient over the whole range of gates, its limits where a factor overflows."""
    low, big = torch.finfo(BF16).tiny, torch.finfo(BF16).max
    v = [0.0, -0.0, low, 1e-20, 1e-3, 0.5, 1.0, 3.0, 8.0, 30.0, 88.0, 100.0, 1e4, 1e10, 1e19, 1e30, big]
    g = torch.tensor(v + [-t for t in v] + [-1.5, 2.5, -6.0, 6.0, -89.0, 7.5], device="cuda").to(BF16)
    F, K = g.numel(), 8
    assert F % 8 == 0
    pre = torch.cat([g, torch.full_like(g, 2.0)])[None].repeat(3, 1).contiguous()
    d = torch.ones(3, F, dtype=BF16, device="cuda")
    dp = torch.empty_like(pre)
    w, x = torch.zeros(2 * F, K, dtype=BF16, device="cuda"), torch.zeros(3, K, dtype=BF16, device="cuda")
    L.gated_matmul_bf16_backward(x, w, act, pre, d, dp)
    gd = f64(g)
    slope, value = np.where(gd > 20, 1.0, 0.0), np.where(gd > 0, gd, 0.0)   # their limits
    near = np.abs(gd) < 100
    sl, va = ref.act_slope(np.where(near, gd, 0.0), act)
    slope, value = np.where(near, sl, slope), np.where(near, va, value)
    got = f64(dp)
    want = np.concatenate([2 * slope, value])[None]
    # 100 terms of |z| U and a rounding; below 1e-30 the reciprocal's flush to zero counts
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 2e-4) + 1e-30).all(), np.abs(got - want).max()


def train_and_serve(L, seed=5):  # noqa: F811
    """A forward and backward pass of a dense expert, and a pass with adapters: what runs, and its results."""
    from expert_ffn_amd.layer import Adapters, DenseExpertBf16
    T, H, FF, n, R = 77, 256, 192, 6, 16
    g = gen(seed)
    blob = torch.zeros(L.expert_bytes(L.W_BF16, H, FF), dtype=torch.uint8, device="cuda")
    L.pack_expert(L.W_BF16, normal(g, 2 * FF, H, dtype=BF16, scale=H ** -0.5), normal(g, H, FF, dtype=BF16, scale=FF ** -0.5), blob)
    ad = Adapters(n, R, H, FF)
    for i in range(n - 1):   # the last slot stays empty
        r = (5, 8, 16, 1, 12)[i]
        ad.load(i, normal(g, 2, r, H, dtype=BF16, scale=H ** -0.5), normal(g, 2 * FF, r, dtype=BF16, scale=0.3),
                normal(g, r, FF, dtype=BF16, scale=FF ** -0.5), normal(g, H, r, dtype=BF16, scale=0.3), 0.5 + i)
    e = DenseExpertBf16(blob, H, FF, act=1, adapters=ad)
    x, dy = normal(g, T, H, dtype=BF16), normal(g, T, H, dtype=BF16)
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    new = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")
    o = dict(hid=new(T, FF), y=new(T, H), pre=new(T, 2 * FF), dhid=new(T, FF), dpre=new(T, 2 * FF), dx=new(T, H),
             dw13=new(2 * FF, H, dt=F32), dw2=new(H, FF), low=new(T, 2 * R), hid_a=new(T, FF), y_a=new(T, H))

    def run(stream=None):
        e.run(x, o["hid"], o["y"], pre=o["pre"], stream=stream)
        e.backward(x, o["pre"], o["hid"], dy, o["dhid"], o["dpre"], dx=o["dx"], dw13=o["dw13"], dw2=o["dw2"], stream=stream)
        e.run(x, o["hid_a"], o["y_a"], low=o["low"], adapter_ids=ids, stream=stream)

    return e, x, dy, ids, o, run


def test_replayed_graph(L):  # noqa: F811
    _, x, _, ids, o, run = train_and_serve(L)
    run()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in o.items()}
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    for i in range(4):
        for v in o.values():
            v.fill_(float(i))
        graph.replay()
        torch.cuda.synchronize()
        for k, v in o.items():
            assert torch.equal(v, want[k]), (i, k)
        run()                                        # eager work between the replays
        torch.cuda.synchronize()
    # other rows and ids in the same buffers
    x.copy_(x.flip(0).clone())
    ids.copy_(ids.flip(0).clone())
    graph.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in o.items()}
    run()
    torch.cuda.synchronize()
    for k, v in o.items():
        assert torch.equal(v, got[k]), k
    # rows depend on their own token (with adapters the order of a row's sums depends on the tokens around it)
    for k in ("hid", "y", "pre"):
        assert torch.equal(o[k], want[k].flip(0)), k


def test_two_streams(L):  # noqa: F811
    """Two experts' passes on two streams at once, each given by argument or as the current one."""
    sets = [train_and_serve(L, seed) for seed in (1, 2)]
    want = []
    for *_, o, run in sets:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in o.items()})
        for v in o.values():
            v.zero_()
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        sets[0][5](st[0])
        with torch.cuda.stream(st[1]):
            sets[1][5]()
    torch.cuda.synchronize()
    for (*_, o, _), w in zip(sets, want):
        for k, v in o.items():
            assert torch.equal(v, w[k]), k


def test_repeated_runs_are_equal(L):  # noqa: F811
    """Sums have a fixed order: the same bits every time."""
    for T, F, K in ((77, 704, 1424), (1030, 2112, 328)):
        g = gen(T)
        x, w = normal(g, T, K, dtype=BF16), normal(g, 2 * F, K, dtype=BF16, scale=K ** -0.5)
        d = normal(g, T, F, dtype=BF16)
        got = []
        for _ in range(4):
            out, pre = torch.empty(T, F, device="cuda"), torch.empty(T, 2 * F, dtype=BF16, device="cuda")
            dx, dw = torch.empty(T, K, device="cuda"), torch.empty(2 * F, K, device="cuda")
            L.gated_matmul_bf16(x, w, 0, out, pre=pre)
            L.gated_matmul_bf16_backward(x, w, 0, pre, d, torch.empty_like(pre), dx=dx, dw=dw)
            got.append((out, pre, dx, dw))
        torch.cuda.synchronize()
        for o in got[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, got[0]))


def test_expert_with_adapters_against_64_bits(L):  # noqa: F811
    """DenseExpertBf16 with adapters: each product against 64 bits on what the one before it stored."""
    e, x, dy, ids, o, run = train_and_serve(L)
    run()
    torch.cuda.synchronize()
    ad, H, FF, U = e.adapters, e.H, e.FF, block_ref.U
    none = lambda b: torch.zeros_like(b)
    for xin, w, a, b, halves, out in ((x, e.w13, ad.a13, ad.b13, 2, o["hid_a"]), (o["hid_a"], e.w2, ad.a2[:, None], ad.b2, 1, o["y_a"])):
        K, R = xin.shape[1], ad.R
        low, _ = ref.adapters(xin, ids, a, none(b), ad.scale, ad.ranks, halves)
        mag, _ = ref.adapters(xin.abs(), ids, a.abs(), none(b), ad.scale.abs(), ad.ranks, halves)
        s = torch.empty(x.shape[0], halves * R, dtype=BF16, device="cuda")
        L.adapter_shrink(xin, ids, a if halves == 2 else a[:, 0], ad.scale, s, ranks=ad.ranks)
        # K additions and the scale, at most two half steps each, then the rounding to bf16
        e_low = f64(mag) * 2 * (K + 2) * U
        close(f64(s), f64(low), e_low + half_step(BF16) * (np.abs(f64(low)) + e_low), "s")
        v, m = (xin.to(F64) @ w.to(F64).t().contiguous()), xin.to(F64).abs() @ w.to(F64).abs().t().contiguous()
        N = w.shape[0] // halves
        for k in range(ad.n):
            rows = (ids == k).nonzero()[:, 0]
            for h in range(halves):
                c = slice(h * N, (h + 1) * N)
                sk, bk = s[rows, h * R:(h + 1) * R].to(F64), b[k, c].to(F64).t().contiguous()
                v[rows, c] += sk @ bk
                m[rows, c] += sk.abs() @ bk.abs()
        dv = f64(m) * 2 * (K + R + 8) * U
        v = f64(v)
        if halves == 2:
            g, u, dg, du = v[:, :N], v[:, N:], dv[:, :N], dv[:, N:]
            want, bound = block_ref.gated(g, u, e.act)
            # |act'| <= 1.13 and |act(g)| <= |g|
            bound = bound + 1.13 * dg * (np.abs(u) + du) + (np.abs(g) + dg) * du
        else:
            want, bound = v, dv
        close(f64(out), want, bound + half_step(BF16) * (np.abs(want) + bound), "out")


def test_block_with_a_bf16_expert(L):  # noqa: F811
    """MoeBlock with a DenseExpertBf16: the dense rows are the expert's on the block's x, with and without adapters,
    and the block is otherwise that of the routed experts and these rows."""
    import synth
    from gpu_common import build_pool
    from expert_ffn_amd.layer import MoeBlock, MoeLayer
    e, _, _, _, _, _ = train_and_serve(L)
    E, k, H, FF, T = 16, 4, 256, 128, 33
    slot_of = np.arange(E, dtype=np.int32)
    pool, sb = build_pool(0, 0, E, H, FF, L.W_BF16, slot_of)
    g = gen(9)
    w_in, w_post, wr = (0.1 * normal(g, H)).to(BF16), (0.1 * normal(g, H)).to(BF16), normal(g, E, H, scale=H ** -0.5)
    block = lambda dense: MoeBlock(MoeLayer(E, k, H, FF, L.W_BF16, T + 2).bind(pool, sb, torch.from_numpy(slot_of).cuda()), w_in, wr,
                                   w_post=w_post, w_offset=1.0, dense=dense)
    h = normal(g, T, H, dtype=BF16, scale=2.0)
    ids = torch.randint(-1, e.adapters.n, (T,), generator=g, device="cuda").to(torch.int32)
    b = block(e)
    rows = []
    for a in (None, ids):
        out = torch.empty_like(h)
        b.run(h, out, adapter_ids=a)
        hid, y, low = torch.empty(T, e.FF, dtype=BF16, device="cuda"), torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(
            T, 2 * e.adapters.R, dtype=BF16, device="cuda")
        e.run(b.x[:T], hid, y, low=low, adapter_ids=a)
        torch.cuda.synchronize()
        assert torch.equal(b.yd[:T], y)
        want = torch.empty_like(h)
        Lr = b.layer
        L.norm_out(h, want, w_post, 1e-6, out_routes=Lr.out_routes[:T * k], topk_w=Lr.topk_w[:T], route_pos=Lr.route_pos[:T * k], y=y,
                   w_offset=1.0)
        assert torch.equal(out, want)
        rows.append(y)
    assert not torch.equal(*rows)
    plain = torch.empty_like(h)
    block(None).run(h, plain)
    assert not torch.equal(plain, out)
    with pytest.raises(ValueError, match="no adapters"):
        block(None).run(h, plain, adapter_ids=ids)
    with pytest.raises(ValueError, match="need low"):
        e.run(h, hid, y, adapter_ids=ids)

"""The whole block (MoeBlock: norm, scored routing, routed and dense experts, combine,
norm, gate, residual, next norm) on the GPU: every link against the 64-bit
definition applied to what the link before it stored, graph replays, other streams,
and matrices whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import block_ref as ref
import synth
from block_ref import U, f64, half_step
from gpu_common import TOL, build_pool
from test_gpu_block import close

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def L():
    import expert_ffn_amd as lib
    lib.lib()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def make_block(lib, *, fmt, T_max, E=16, k=4, H=256, FF=128, FFd=192, seed=0, drop=True, ht=BF16, n_group=4,
               topk_group=2, dense=True, gate="channel"):
    from expert_ffn_amd.layer import DenseExpert, MoeBlock, MoeLayer
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    slot_of = np.arange(E, dtype=np.int32)[::-1].copy()
    if drop:
        slot_of[[2, 7]] = -1
    pool, sb = build_pool(seed, 0, E, H, FF, fmt, slot_of)
    layer = MoeLayer(E, k, H, FF, fmt, T_max).bind(pool, sb, torch.from_numpy(slot_of).cuda())
    d = None
    if dense:
        w13, w2 = synth.expert_weights(seed, 1, 0, H, FFd)
        blob = torch.zeros(lib.expert_bytes(lib.W_INT8_ROW, H, FFd), dtype=torch.uint8, device="cuda")
        lib.pack_expert(lib.W_INT8_ROW, torch.from_numpy(w13.view(np.int16)).cuda(), torch.from_numpy(w2.view(np.int16)).cuda(),
                        blob)
        d = DenseExpert(blob, H, FFd)
    gt = {None: None, "channel": 0.5 + torch.rand(H, generator=g, device="cuda"),
          "token": 0.5 + torch.rand(T_max, 1, generator=g, device="cuda")}[gate]
    w_in, w_post, w_next = ((0.1 * n(H)).to(BF16) for _ in range(3))
    return MoeBlock(layer, w_in, n(E, H) / H ** 0.5, w_post=w_post, eps=EPS, w_offset=1.0, dense=d, gate=gt,
                    block_scale=0.9, res_scale=1.1, w_next=w_next, score=lib.SCORE_SIGMOID, bias=0.1 * n(E),
                    n_group=n_group, topk_group=topk_group, group_rank=lib.GROUP_TOP2, route_scale=2.5), slot_of


def rows(T, H, seed, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(T, H, generator=g, device="cuda") * 2).to(dtype)


def check_links(lib, b, slot_of, h, h_out, x_next):
    T, Lr = h.shape[0], b.layer
    k = Lr.k
    # norm before
    want, r = ref.norm_in(f64(h), f64(b.w_in), b.w_offset, EPS)
    x = b.x[:T]
    close(f64(x), want, np.abs(want) * (ref.NORM_U + half_step(BF16) * (1 + ref.NORM_U)) + 1e-37, "x")
    # router product (fp32 sums of H terms), then the choice on the logits as stored
    lg = f64(x) @ f64(b.w_router).T
    mag = np.abs(f64(x)) @ np.abs(f64(b.w_router)).T
    close(f64(b.logits[:T]), lg, Lr.H * U * mag, "logits")
    rt = b.routing
    ids, w = ref.route_score(f64(b.logits[:T]), k, rt["score"], f64(rt["bias"]), rt["n_group"], rt["topk_group"],
                             rt["group_rank"] == lib.GROUP_TOP2, rt["renorm"], rt["scale"])
    assert np.array_equal(Lr.topk_ids[:T].cpu().numpy(), ids)
    close(f64(Lr.topk_w[:T]), w, U * (1 + 1e-6) * np.abs(w), "weights")
    pos = Lr.route_pos[:T * k].cpu().numpy().reshape(T, k)
    assert np.array_equal(pos >= 0, slot_of[ids] >= 0)
    y = None
    if b.dense is not None:
        d = b.dense
        q, s = ref.codes(ref.unnormed(h.float().cpu().numpy(), b.w_in.float().cpu().numpy(), b.w_offset))
        assert np.array_equal(b.xq[:T].cpu().numpy(), q)
        close(f64(b.xs[:T]), s * r[:, 0], s * r[:, 0] * ref.NORM_U, "scales")
        v, _ = ref.matmul_i8(q, f64(b.xs[:T]), d.w13.cpu().numpy(), f64(d.s13))
        hid, bound = ref.gated(v[:, :d.FF], v[:, d.FF:], 0)
        close(f64(b.hid[:T]), hid, bound + half_step(BF16) * (np.abs(hid) + bound), "dense hidden")
        q, s = ref.codes(b.hid[:T].float().cpu().numpy())
        assert np.array_equal(b.hq[:T].cpu().numpy(), q) and np.array_equal(b.hs[:T].cpu().numpy(), s)
        v, bound = ref.matmul_i8(q, s, d.w2.cpu().numpy(), f64(d.s2))
        close(f64(b.yd[:T]), v, bound + half_step(BF16) * (np.abs(v) + bound), "dense rows")
        y = f64(b.yd[:T])
    gate = None
    if b.gate is not None:
        gate = f64(b.gate[:T]) if b.gate.dim() == 2 else f64(b.gate)
    want, bound = ref.norm_out(f64(h), np.nan_to_num(f64(Lr.out_routes[:T * k])), f64(Lr.topk_w[:T]), pos, y, f64(b.w_post),
                               b.w_offset, EPS, gate, np.float64(np.float32(b.block_scale)),
                               np.float64(np.float32(b.res_scale)))
    close(f64(h_out), want, bound + half_step(h.dtype) * (np.abs(want) + bound), "h_out")
    want, _ = ref.norm_in(f64(h_out), f64(b.w_next), b.w_offset, EPS)
    close(f64(x_next), want, np.abs(want) * (ref.NORM_U + half_step(BF16) * (1 + ref.NORM_U)) + 1e-37, "x_next")


@pytest.mark.parametrize("fmt,T,ht,dense,gate", [(1, 1, BF16, True, "channel"), (2, 16, F32, True, "token"),
                                                 (2, 77, BF16, True, None), (0, 33, F32, False, "channel"),
                                                 (1, 300, BF16, True, "token")])
def test_block_links(L, fmt, T, ht, dense, gate):
    b, slot_of = make_block(L, fmt=fmt, T_max=T + 3, dense=dense, gate=gate, seed=fmt + T)
    h = rows(T, 256, T, ht)
    ho = torch.full((T + 1, 256), 3.0, dtype=ht, device="cuda")
    out, xn = b.run(h, ho[:T])
    torch.cuda.synchronize()
    assert out.data_ptr() == ho.data_ptr() and (ho[T] == 3.0).all()
    check_links(L, b, slot_of, h, ho[:T], xn)
    # in place, twice: the same bits
    for _ in range(2):
        h2 = h.clone()
        _, xn2 = b.run(h2, h2)
        assert torch.equal(h2, ho[:T]) and torch.equal(xn2, xn)


def test_block_against_the_oracle(L):
    """The routed experts' share of the block against the oracle's layer on the x the block stored."""
    from gpu_common import oracle_layer
    T, fmt = 24, 1
    b, slot_of = make_block(L, fmt=fmt, T_max=T, dense=False, gate=None, seed=3)
    h = rows(T, 256, 5, F32)
    ho = torch.empty_like(h)
    b.run(h, ho)
    Lr = b.layer
    r = oracle_layer(3, 0, Lr.E, Lr.k, Lr.H, Lr.FF, fmt, 0, b.logits[:T].cpu().numpy(), b.x[:T].float().cpu().numpy(), slot_of,
                     np.arange(T), routes_in=(Lr.topk_ids[:T].cpu().numpy(), Lr.topk_w[:T].cpu().numpy()))
    want, _ = ref.norm_out(f64(h), None, None, None, np.asarray(r["y"], np.float64), f64(b.w_post), b.w_offset, EPS, None,
                           b.block_scale, b.res_scale)
    # y is within TOL of each row's largest |y| and the norm divides by the row's rms, so n moves by at most
    # TOL max|y| / rms (1 + max|y| / rms ...): twice that bounds both terms
    y = np.asarray(r["y"], np.float64)
    rms = np.sqrt((y * y).mean(1, keepdims=True) + EPS)
    peak = np.abs(y).max(1, keepdims=True) / rms
    bound = 0.9 * TOL[fmt] * peak * (1 + np.abs(y) / rms) * np.abs(1 + f64(b.w_post)) * 1.1 + 1e-4
    close(f64(ho), want, bound, "h_out")


def test_block_smaller_batches_and_refusals(L):
    b, slot_of = make_block(L, fmt=2, T_max=100, seed=9)
    for T in (100, 1, 64, 65, 0):
        h = rows(T, 256, 40 + T)
        ho = torch.empty_like(h)
        out, xn = b.run(h, ho)
        torch.cuda.synchronize()
        assert out.shape == (T, 256) and xn.shape == (T, 256)
        if T:
            check_links(L, b, slot_of, h, ho, xn)
    with pytest.raises(ValueError, match="T_max"):
        b.run(rows(101, 256, 1), torch.empty(101, 256, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("T", [16, 100])
def test_block_captured_and_replayed(L, T):
    """A captured run against eager runs of the same inputs, several replays with eager work between them."""
    b, _ = make_block(L, fmt=2, T_max=T, seed=T)
    other, _ = make_block(L, fmt=2, T_max=T, seed=T)     # same weights, buffers of its own
    h = rows(T, 256, 1)
    ho = torch.empty_like(h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run(h, ho)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _, xn = b.run(h, ho)
    for i in range(4):
        h.copy_(rows(T, 256, 10 + i))
        want = torch.empty_like(h)
        _, wx = other.run(h, want)
        ho.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ho, want) and torch.equal(xn, wx), f"replay {i} differs"


def test_blocks_on_two_streams(L):
    """Two blocks at once on streams of their own, against the same runs one after the other."""
    T = 48
    blocks = [make_block(L, fmt=1, T_max=T, seed=20 + i)[0] for i in range(2)]
    hs = [rows(T, 256, 30 + i) for i in range(2)]
    want = []
    for b, h in zip(blocks, hs):
        o = torch.empty_like(h)
        _, xn = b.run(h, o)
        want.append((o, xn.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(h) for h in hs]
    for rep in range(10):
        for b in blocks:
            b.x_next.fill_(0)
        torch.cuda.synchronize()
        for b, h, o, s in zip(blocks, hs, outs, streams):
            b.run(h, o, stream=s) if rep % 2 else None
            if not rep % 2:
                with torch.cuda.stream(s):
                    b.run(h, o)
        torch.cuda.synchronize()
        for o, b, (wo, wx) in zip(outs, blocks, want):
            assert torch.equal(o, wo) and torch.equal(b.x_next[:T], wx)


def test_offsets_past_32_bits(L):
    """Rows more than 2^31 elements and 2^32 bytes from the first one."""
    big = torch.empty(5 << 30, dtype=torch.int8, device="cuda")
    # weights: 2100 rows 2^21 bytes apart
    N, K, T = 2100, 64, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    wq = big[:(N << 21)].view(N, 1 << 21)[:, :K]
    wq.copy_(torch.randint(-127, 128, (N, K), generator=g, device="cuda"))
    xq = torch.randint(-127, 128, (T, K), generator=g, device="cuda").to(torch.int8)
    out = torch.empty(T, N, device="cuda")
    one = torch.ones(N, device="cuda")
    L.matmul_i8(xq, one[:T], wq, one, out)
    assert torch.equal(out.cpu().double(), xq.cpu().double() @ wq.cpu().double().T)
    # tokens: the same matrix as the activations, outputs 40000 elements apart
    Tb = N
    outb = torch.empty(Tb, 8, device="cuda")
    L.matmul_i8(wq, one, xq.repeat(2, 1)[:8].contiguous(), one[:8], outb)
    assert torch.equal(outb.cpu().double(), wq.cpu().double() @ xq.repeat(2, 1)[:8].cpu().double().T)
    # outputs: 66000 rows 40000 bf16 apart (2.6e9 elements)
    To = 66000
    o = big.view(torch.bfloat16)[:(To - 1) * 40000 + 32].as_strided((To, 32), (40000, 1))
    xs = torch.randint(-127, 128, (To, 16), generator=g, device="cuda").to(torch.int8)
    ws = torch.randint(-127, 128, (32, 16), generator=g, device="cuda").to(torch.int8)
    ones = torch.ones(To, device="cuda")
    L.matmul_i8(xs, ones, ws, one[:32], o)
    want = (xs.float() @ ws.float().t()).to(BF16)
    assert torch.equal(o, want)
    # norms: rows read and written there
    x = torch.empty(To, 32, dtype=BF16, device="cuda")
    L.norm_in(o, None, EPS, x=x)
    ref_x, _ = ref.norm_in(f64(want), None, 0, EPS)
    close(f64(x), ref_x, np.abs(ref_x) * (ref.NORM_U + half_step(BF16) * 1.001) + 1e-37, "x")
    L.norm_out(x, o, None, EPS, y=x, res_scale=0.0, block_scale=2.0)
    assert torch.equal(o, (2 * x.float()).to(BF16))
    # logits: rows there
    lg = o[:, :8]
    ids = torch.empty(To, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(To, 2, device="cuda")
    L.route_score_topk(lg, 2, ids, w)
    want_ids, _ = ref.route_score(f64(lg), 2, 0)
    assert np.array_equal(ids.cpu().numpy(), want_ids)


@pytest.mark.parametrize("T,k", [(5461, 3), (4096, 4), (4200, 10)])   # 2 GiB less one row, 2 GiB, 5.1 GiB of routes
def test_norm_out_far_routes(L, T, k):
    H, R = 32768, T * k
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    routes = torch.empty(R, H, device="cuda")
    pos = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    tw = torch.full((T, k), float("nan"), device="cuda")
    rows = [(0, 0, R - 1), (1, 1, R // 2), (T - 1, 0, 0), (T - 1, k - 1, R - 2), (T // 2, 2, R - 3)]
    for t, j, r in rows:
        routes[r] = torch.randn(H, generator=g, device="cuda")
        pos[t, j], tw[t, j] = r, 0.5 + j
    h = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    ho = torch.empty_like(h)
    L.norm_out(h, ho, None, EPS, out_routes=routes, topk_w=tw, route_pos=pos)
    want = h.clone()
    for t in sorted({t for t, _, _ in rows}):
        b = torch.zeros(H, device="cuda", dtype=torch.float64)
        for t2, j, r in rows:
            if t2 == t:
                b += (0.5 + j) * routes[r].double()
        want[t] = 0
        # two products and their sum, then the residual: four roundings in 32 bits and the stored one
        full = h[t].double() + b
        assert ((ho[t].double() - full).abs() <= half_step(BF16) * 1.001 * full.abs() + 8 * U * (b.abs() + h[t].double().abs() + 4)).all()
    got = ho.clone()
    got[sorted({t for t, _, _ in rows})] = 0
    assert torch.equal(got, want)


def test_router_score_topk(L):
    """The router's product and the scored top-k on its logits."""
    for T, E, H, dt in ((1, 128, 2816, BF16), (17, 60, 192, F32), (130, 256, 704, BF16), (300, 257, 64, F32)):
        g = torch.Generator(device="cuda")
        g.manual_seed(T)
        x = torch.randn(T, H, generator=g, device="cuda").to(dt)
        wr = torch.randn(E, H, generator=g, device="cuda") / H ** 0.5
        b = 0.1 * torch.randn(E, generator=g, device="cuda")
        k = 6
        ws = torch.empty(L.router_ws_bytes(T, H, E), dtype=torch.uint8, device="cuda")
        lg = torch.empty(T, E, device="cuda")
        ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        w = torch.empty(T, k, device="cuda")
        L.router_score_topk(x, wr, k, lg, ws, ids, w, score=L.SCORE_SIGMOID, bias=b, scale=1.5)
        l2 = torch.empty_like(lg)
        i2, w2 = torch.empty_like(ids), torch.empty_like(w)
        L.router_topk(x, wr, k, l2, ws, i2, w2)
        assert torch.equal(lg, l2), "logits differ from router_topk's"
        want_ids, want_w = ref.route_score(f64(lg), k, 1, f64(b), scale=1.5)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        close(f64(w), want_w, U * (1 + 1e-6) * np.abs(want_w), "weights")

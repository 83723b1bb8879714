"""The operators of the transformer block around the routed expert FFN, as cases to
measure: routing by scores with a balance bias and expert groups, the norms before
and after the block, and the 8-bit integer product of a dense (shared) expert.

Each case runs in two ways on the same inputs: `own` false, its plain form (elementary
torch operations in 32 bits, 64 for the choice of experts); `own` true, the library.
Sizes: the 128-expert top-8 layer of hidden size 2816 and expert size 704 that the
benchmark runs (a dense expert is three of those wide), and generic ones.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a decode step's router: a batch of 16 sequences, one token each
        dict(name="route_decode", op="route", T=16, E=128, k=8, G=1, keep=1, score="softmax", rank="max", bias=True,
             scale=1.0, dt="f32"),
        # a prefill chunk with grouped experts, sigmoid scores and a balance bias
        dict(name="route_chunk_grouped", op="route", T=1024, E=256, k=8, G=8, keep=4, score="sigmoid", rank="top2",
             bias=True, scale=2.5, dt="f32"),
        # many sequences' prompts at once, 16-bit logits (equal ones occur), an expert count that is no power of two
        dict(name="route_long_ragged", op="route", T=16383, E=160, k=6, G=8, keep=3, score="softmax", rank="max",
             bias=False, scale=1.0, dt="bf16"),
        # the norm before the block of a decode step
        dict(name="norm_in_decode", op="norm_in", T=16, H=2816, h="bf16", x="bf16", offset=1.0),
        # the norm over long prompts with a 32-bit residual stream
        dict(name="norm_in_long", op="norm_in", T=8191, H=4104, h="f32", x="bf16", offset=0.0),
        # the end of a decode step's block: combine, dense expert's rows, norm, gate, residual, next norm
        dict(name="norm_out_decode", op="norm_out", T=16, H=2816, k=8, routes="f32", y=True, h="bf16", gate="channel",
             drop=0.0, offset=1.0),
        # the end of a prefill chunk's block, some routes on experts that are not resident
        dict(name="norm_out_chunk", op="norm_out", T=1024, H=2816, k=8, routes="f32", y=True, h="bf16", gate="channel",
             drop=0.1, offset=0.0),
        # one sequence's next token: norm, 8-bit codes and the product with a dense matrix
        dict(name="linear_one_token", op="linear", T=1, K=2816, N=5632, pre="norm", gated=False, out="bf16"),
        # a decode batch through a dense expert's gate and up projections, codes from the rows
        dict(name="gated_decode", op="linear", T=16, K=2816, N=2112, pre="quant", gated=True, out="bf16"),
        # a ragged batch: odd token and channel counts, 32-bit outputs
        dict(name="linear_ragged", op="linear", T=77, K=1424, N=2819, pre="codes", gated=False, out="f32"),
        # a prefill chunk through the dense expert's gate and up projections
        dict(name="gated_chunk", op="linear", T=1024, K=2816, N=2112, pre="codes", gated=True, out="bf16"),
        # long prompts through a large dense matrix
        dict(name="linear_long", op="linear", T=8192, K=4096, N=8192, pre="codes", gated=False, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm_in", "norm_out", "linear", "linear"])
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8, 10])
        size = rng.randint(max(1, 8 // G), 512 // G)
        E = G * size
        keep = rng.randint(1, G)
        k = rng.randint(1, min(32, keep * size, 10))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, G=G, keep=keep, score=rng.choice(["softmax", "sigmoid"]),
                    rank=rng.choice(["max", "top2"]), bias=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dt=rng.choice(["f32", "bf16"]))
    if op == "norm_in":
        H = 8 * _log(rng, 8, 1024)
        return dict(op=op, T=_log(rng, 1, min(16384, (8191 * 4104) // H)), H=H, h=rng.choice(["bf16", "f32"]),
                    x=rng.choice(["bf16", "f32"]), offset=rng.choice([0.0, 1.0]))
    if op == "norm_out":
        H = 8 * _log(rng, 8, 1024)
        k = rng.randint(1, 10)
        return dict(op=op, T=_log(rng, 1, max(2, (1024 * 2816 * 8) // (H * k))), H=H, k=k,
                    routes=rng.choice(["bf16", "f32"]), y=rng.random() < 0.7, h=rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["none", "channel", "token"]), drop=rng.choice([0.0, 0.1, 0.9]),
                    offset=rng.choice([0.0, 1.0]))
    K = 16 * _log(rng, 8, 512)
    N = _log(rng, 64, 8192)
    gated = rng.random() < 0.4
    most = 8192 * 4096 * 8192 // (K * N * (2 if gated else 1))
    return dict(op=op, T=_log(rng, 1, max(1, min(8192, most))), K=K, N=N,
                pre=rng.choice(["norm", "quant", "codes"]), gated=gated, out=rng.choice(["bf16", "f32"]))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 13)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    def empty(*shape, dtype):
        return torch.empty(shape, device=dev, dtype=dtype)

    s = dict(case)
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        # an uneven popularity of the experts on top of unit-variance logits
        pop = -1.1 * torch.log(torch.randperm(E, generator=g, device=dev).float() + 1.0)
        s["logits"] = (normal(T, E) + 0.5 * pop).to(DT[case["dt"]])
        s["b"] = 0.1 * normal(E) if case["bias"] else None
        s["ids"], s["w"] = empty(T, k, dtype=torch.int32), empty(T, k, dtype=torch.float32)
        return s
    if op == "linear":
        K, N = case["K"], case["N"]
        rows = 2 * N if case["gated"] else N
        s["wq"], s["sw"] = _codes(0.02 * normal(rows, K))
        s["out"] = empty(T, N, dtype=DT[case["out"]])
        s["h"] = (normal(T, K) * (0.5 + uniform(T, 1))).to(torch.bfloat16)
        s["w_in"] = (1.0 + 0.1 * normal(K)).to(torch.bfloat16)
        if case["pre"] == "codes":
            s["xq"], s["sx"] = _codes(s["h"].float())
        else:
            s["xq"], s["sx"] = empty(T, K, dtype=torch.int8), empty(T, dtype=torch.float32)
        return s
    H = case["H"]
    s["h"] = (normal(T, H) * (0.5 + 4.0 * uniform(T, 1))).to(DT[case["h"]])
    s["w_in"] = (1.0 - case["offset"] + 0.1 * normal(H)).to(torch.bfloat16)
    if op == "norm_in":
        s["xo"] = empty(T, H, dtype=DT[case["x"]])
        return s
    k = case["k"]
    R = T * k
    s["o"] = (0.3 * normal(R, H)).to(DT[case["routes"]])
    pos = torch.randperm(R, generator=g, device=dev).to(torch.int32)
    s["pos"] = torch.where(uniform(R) < case["drop"], torch.full_like(pos, -1), pos).view(T, k)
    e = torch.exp(normal(T, k))
    s["w"] = e / e.sum(1, keepdim=True)
    s["y"] = (0.5 * normal(T, H)).to(torch.bfloat16) if case["y"] else None
    s["w_post"] = (1.0 - case["offset"] + 0.1 * normal(H)).to(torch.bfloat16)
    s["gate"] = {"none": None, "channel": 0.5 + uniform(1, H), "token": uniform(T, 1)}[case["gate"]]
    s["ho"], s["xo"] = empty(T, H, dtype=DT[case["h"]]), empty(T, H, dtype=torch.bfloat16)
    return s


def _codes(u):
    """8-bit codes and the scale of each row: a = max |u|, scale = a / 127, codes = rint(u / scale), all in fp32."""
    sc = u.abs().amax(1, keepdim=True) / 127.0
    q = torch.where(sc > 0, torch.round(u / sc), torch.zeros_like(u)).clamp_(-127, 127)
    return q.to(torch.int8), sc[:, 0].contiguous()


def _act(g):
    return g * 0.5 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _rms(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _route_plain(s):
    l = s["logits"].double()   # the choice stands next to borders: 64 bits
    T, E = l.shape
    G, size = s["G"], s["E"] // s["G"]
    if s["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    c = p if s["b"] is None else p + s["b"].double()
    if s["keep"] < G:
        cg = c.view(T, G, size)
        if s["rank"] == "max" or size == 1:
            gs = cg.amax(2)
        else:
            gs = cg.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = torch.where(kept[:, :, None], cg, torch.full_like(cg, -math.inf)).view(T, E)
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * s["scale"]
    return {"ids": ids.to(torch.int32), "w": w.float()}


def _norm_out_plain(s):
    pos, w = s["pos"].long(), s["w"]
    ok = (pos >= 0)[:, :, None]
    rows = s["o"][pos.clamp_min(0)].float()
    b = torch.where(ok, rows * w[:, :, None], torch.zeros_like(rows)).sum(1)
    if s["y"] is not None:
        b = b + s["y"].float()
    n = b * _rms(b) * (s["offset"] + s["w_post"].float())
    if s["gate"] is not None:
        n = n * s["gate"]
    ho = (s["h"].float() + n).to(s["h"].dtype)
    hf = ho.float()
    x = (hf * _rms(hf) * (s["offset"] + s["w_in"].float())).to(torch.bfloat16)
    return {"h": ho, "x": x}


def _linear_plain(s):
    xq, sx = s["xq"], s["sx"]
    if s["pre"] == "norm":
        hf = s["h"].float()
        xq, sx = _codes(hf * s["w_in"].float())
        sx = sx * _rms(hf)[:, 0]
    elif s["pre"] == "quant":
        xq, sx = _codes(s["h"].float())
    v = (xq.float() @ s["wq"].float().t()) * sx[:, None] * s["sw"][None, :]
    if s["gated"]:
        v = _act(v[:, :s["N"]]) * v[:, s["N"]:]
    return v.to(s["out"].dtype)


def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "route":
        return _route_plain(s)
    if op == "norm_in":
        hf = s["h"].float()
        return (hf * _rms(hf) * (s["offset"] + s["w_in"].float())).to(s["xo"].dtype)
    if op == "norm_out":
        return _norm_out_plain(s)
    return _linear_plain(s)


def _run_own(s):
    import expert_ffn_amd as lib
    op = s["op"]
    if op == "route":
        lib.route_score_topk(s["logits"], s["k"], s["ids"], s["w"],
                             score=lib.SCORE_SOFTMAX if s["score"] == "softmax" else lib.SCORE_SIGMOID,
                             bias=s["b"], n_group=s["G"], topk_group=s["keep"],
                             group_rank=lib.GROUP_MAX if s["rank"] == "max" else lib.GROUP_TOP2, scale=s["scale"])
        return {"ids": s["ids"], "w": s["w"]}
    if op == "norm_in":
        lib.norm_in(s["h"], s["w_in"], EPS, x=s["xo"], w_offset=s["offset"])
        return s["xo"]
    if op == "norm_out":
        lib.norm_out(s["h"], s["ho"], s["w_post"], EPS, out_routes=s["o"], topk_w=s["w"], route_pos=s["pos"],
                     y=s["y"], gate=s["gate"], w_next=s["w_in"], x=s["xo"], w_offset=s["offset"])
        return {"h": s["ho"], "x": s["xo"]}
    if s["pre"] == "norm":
        lib.norm_in(s["h"], s["w_in"], EPS, xq=s["xq"], xq_scale=s["sx"])
    elif s["pre"] == "quant":
        lib.quantize_tokens(s["h"], s["xq"], s["sx"])
    if s["gated"]:
        lib.gated_matmul_i8(s["xq"], s["sx"], s["wq"], s["sw"], lib.ACT_GELU_TANH, s["out"])
    else:
        lib.matmul_i8(s["xq"], s["sx"], s["wq"], s["sw"], s["out"])
    return s["out"]


def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * SIZE[case["dt"]] + E * 4 * case["bias"] + T * k * 8, "flops": T * E * (4 + k)}
    if op == "linear":
        K, N = case["K"], case["N"]
        rows = 2 * N if case["gated"] else N
        x = T * (K + 4) if case["pre"] == "codes" else T * K * 2 + (K * 2 if case["pre"] == "norm" else 0)
        return {"bytes": x + rows * (K + 4) + T * N * SIZE[case["out"]], "flops": 2 * T * rows * K}
    H = case["H"]
    if op == "norm_in":
        return {"bytes": T * H * (SIZE[case["h"]] + SIZE[case["x"]]) + 2 * H, "flops": 4 * T * H}
    k = case["k"]
    kept = T * k * (1.0 - case["drop"])
    gate = {"none": 0, "channel": 4 * H, "token": 4 * T}[case["gate"]]
    return {"bytes": kept * H * SIZE[case["routes"]] + T * k * 8 + T * H * (2 * case["y"] + 2 * SIZE[case["h"]] + 2)
            + 4 * H + gate, "flops": 2 * kept * H + 10 * T * H}


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    f64 = torch.float64
    if op == "route":
        return _route_exact(s)
    if op == "linear":
        # the 8-bit codes are defined by their 32-bit arithmetic; the product is taken in 64 bits
        N, K = case["N"], case["K"]
        if 2 * T * s["wq"].shape[0] * K > 2e13:
            return None
        xq, sx = s["xq"], s["sx"].to(f64)
        if case["pre"] != "codes":
            u = s["h"].float()
            if case["pre"] == "norm":
                u = u * s["w_in"].float()
            top = u.abs().max(dim=1).values
            step = top / 127.0
            xq = torch.zeros_like(u)
            live = step > 0
            xq[live] = torch.round(u[live] / step[live, None])
            sx = step.to(f64)
            if case["pre"] == "norm":
                sx = sx / (s["h"].to(f64).pow(2).sum(1) / K + EPS).sqrt()
        a = xq.to(f64)
        out = torch.empty((T, s["wq"].shape[0]), dtype=f64, device=a.device)
        for n0 in range(0, out.shape[1], 4096):
            wt = s["wq"][n0:n0 + 4096].to(f64) * s["sw"][n0:n0 + 4096].to(f64)[:, None]
            out[:, n0:n0 + 4096] = torch.mm(a, wt.t().contiguous())
        out *= sx[:, None]
        if case["gated"]:
            g, u = out[:, :N], out[:, N:]
            # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))
            out = g / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g.pow(3)))) * u
        return out
    off = case["offset"]

    def norm(v, w):
        return v / (v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * (off + w.to(f64))

    if op == "norm_in":
        return norm(s["h"].to(f64), s["w_in"])
    b = torch.zeros((T, case["H"]), dtype=f64, device=s["h"].device)
    for j in range(case["k"]):
        p = s["pos"][:, j].long()
        live = (p >= 0).nonzero()[:, 0]
        b[live] += s["w"][live, j].to(f64)[:, None] * s["o"][p[live]].to(f64)
    if s["y"] is not None:
        b += s["y"].to(f64)
    n = norm(b, s["w_post"])
    if s["gate"] is not None:
        n = n * s["gate"].to(f64)
    h = s["h"].to(f64) + n
    # the next norm is that of the residual row as it is stored
    return {"h": h, "x": norm(h.to(s["h"].dtype).to(f64), s["w_in"])}


def _route_exact(s):
    import numpy as np
    l = s["logits"].to(torch.float64).cpu().numpy()
    T, E = l.shape
    G = s["G"]
    if s["score"] == "softmax":
        p = np.exp(l - l.max(1)[:, None])
        p /= p.sum(1)[:, None]
    else:
        p = 1.0 / (1.0 + np.exp(-l))
    c = p.copy() if s["b"] is None else p + s["b"].to(torch.float64).cpu().numpy()[None, :]
    if s["keep"] < G:
        cg = c.reshape(T, G, E // G)
        two = 1 if s["rank"] == "max" else min(2, E // G)
        rank = np.partition(cg, E // G - two, axis=2)[:, :, E // G - two:].sum(2)
        order = np.argsort(-rank, axis=1, kind="stable")
        cg[np.arange(T)[:, None], order[:, s["keep"]:]] = -np.inf
        c = cg.reshape(T, E)
    rows = np.arange(T)
    ids = np.empty((T, s["k"]), np.int32)
    w = np.empty((T, s["k"]))
    for j in range(s["k"]):   # the first of the largest, k times
        best = c.argmax(1)
        ids[:, j], w[:, j] = best, p[rows, best]
        c[rows, best] = -np.inf
    w = w / w.sum(1)[:, None] * s["scale"]
    return {"ids": torch.from_numpy(ids), "w": torch.from_numpy(w)}

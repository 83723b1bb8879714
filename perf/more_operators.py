"""The dense (shared) expert in bf16 beside the routed ones, as cases to measure: the gated
half of a feed-forward block in one kernel (both projections, the activation and the
product) with its backward pass, the plain product's backward pass, and low-rank adapters
of many requests at once beside a shared projection.

Each case runs in two ways on the same inputs: `own` false, its plain form (elementary
torch operations in 32 bits); `own` true, the library.  Sizes: the layer of hidden size
2816 that the benchmark runs (a dense expert is 2112 wide), and generic ones.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one sequence's next token through a dense expert's gate and up projections
        dict(name="gated_one_token", op="gated", T=1, K=2816, F=2112, act="gelu", out="bf16", pre=False),
        # a ragged batch: odd token and channel counts, 32-bit outputs
        dict(name="gated_ragged", op="gated", T=77, K=1424, F=1411, act="silu", out="f32", pre=False),
        # a training step's forward over a few sequences, keeping the pre-activations
        dict(name="gated_train", op="gated", T=4096, K=2816, F=2112, act="gelu", out="bf16", pre=True),
        # its backward over one short sequence
        dict(name="gated_grad_short", op="gated_grad", T=333, K=1424, F=704, act="silu", dw=True),
        # its backward over a chunk, weights frozen (adapters or the layers below are trained)
        dict(name="gated_grad_frozen", op="gated_grad", T=1024, K=2816, F=2112, act="gelu", dw=False),
        # its backward over many sequences in a wide layer
        dict(name="gated_grad_long", op="gated_grad", T=8192, K=4096, F=4096, act="silu", dw=True),
        # the down projection's backward, a ragged batch of the benchmark's layer
        dict(name="grad_ragged", op="grad", T=1001, K=704, N=2816),
        # the down projection's backward over a few sequences
        dict(name="grad_train", op="grad", T=4096, K=2112, N=2816),
        # one sequence's next token through the down projection with its request's adapter
        dict(name="adapters_one_token", op="adapters", T=1, K=2112, N=2816, gated=False, R=16, n=8, mix="tokens",
             none=0.0, uneven=False),
        # a decode batch, each token of another request, through gate and up
        dict(name="adapters_decode", op="adapters", T=16, K=2816, N=2112, gated=True, R=16, n=32, mix="tokens", none=0.1,
             uneven=False),
        # a large decode batch, adapters of several ranks in one pool
        dict(name="adapters_batch", op="adapters", T=129, K=2112, N=2816, gated=False, R=64, n=32, mix="tokens", none=0.2,
             uneven=True),
        # prompts of several requests in one chunk, through gate and up
        dict(name="adapters_prompts", op="adapters", T=2048, K=2816, N=2112, gated=True, R=32, n=24, mix="prompts",
             none=0.1, uneven=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = 8192 * 4096 * 4096   # T K F of the largest listed case


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "grad", "adapters", "adapters"])
    K = 8 * _log(rng, 16, 512)
    if op == "gated":
        F = _log(rng, 64, 4096)
        return dict(op=op, T=_log(rng, 1, min(8192, MOST // (K * F))), K=K, F=F, act=rng.choice(["gelu", "silu"]),
                    out=rng.choice(["bf16", "f32"]), pre=rng.random() < 0.4)
    if op == "gated_grad":
        F = 8 * _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 16, min(8192, MOST // (K * F))), K=K, F=F, act=rng.choice(["gelu", "silu"]),
                    dw=rng.random() < 0.7)
    if op == "grad":
        N = 8 * _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 16, min(8192, MOST // (K * N))), K=K, N=N)
    N, R = _log(rng, 64, 4096), 8 * rng.choice([1, 2, 2, 4, 5, 8, 16])
    T = _log(rng, 1, min(4096, MOST // (K * N)))
    return dict(op=op, T=T, K=K, N=N, gated=rng.random() < 0.5, R=R, n=_log(rng, 1, min(64, 2048 // R)),
                mix="prompts" if T > 64 and rng.random() < 0.7 else "tokens", none=rng.choice([0.0, 0.1, 0.5]),
                uneven=rng.random() < 0.5)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 29)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, device=dev, dtype=dtype)

    s = dict(case)
    op, T, K = case["op"], case["T"], case["K"]
    # activations after a norm, weights that keep their variance
    s["x"] = normal(T, K).to(torch.bfloat16)
    N = case["F"] if "F" in case else case["N"]
    rows = 2 * N if op in ("gated", "gated_grad") or case.get("gated") else N
    s["w"] = (normal(rows, K) / math.sqrt(K)).to(torch.bfloat16)
    if op == "gated":
        s["h"] = empty(T, N, dtype=DT[case["out"]])
        s["p"] = empty(T, 2 * N) if case["pre"] else None
        return s
    if op in ("gated_grad", "grad"):
        s["dy"] = (0.1 * normal(T, N) * (0.5 + uniform(T, 1))).to(torch.bfloat16)
        s["dx"] = empty(T, K)
        s["dweight"] = empty(rows, K) if case.get("dw", True) else None
        if op == "gated_grad":
            s["p"], s["dp"] = normal(T, 2 * N).to(torch.bfloat16), empty(T, 2 * N)
        return s
    n, R, halves = case["n"], case["R"], 2 if case["gated"] else 1
    s["a"] = (normal(n, halves, R, K) / math.sqrt(K)).to(torch.bfloat16)
    s["b"] = (0.2 * normal(n, rows, R)).to(torch.bfloat16)
    if case["uneven"]:   # ranks 8 .. R in steps of 8, smaller ones more often
        s["ranks"] = (8 * torch.ceil(R / 8 * uniform(n) ** 2).clamp_min(1)).to(torch.int32)
    else:
        s["ranks"] = torch.full((n,), R, dtype=torch.int32, device=dev)
    s["scale"] = 2.0 * (0.5 + uniform(n)) / torch.sqrt(s["ranks"].float())
    if case["mix"] == "tokens":
        of = torch.arange(T, device=dev)
    else:   # prompts of uneven lengths: a request begins at about one token in 150, and at the first
        of = torch.cumsum((uniform(T) < 1.0 / 150).long(), 0)
    ids = torch.floor(uniform(T) * n).clamp_max(n - 1).to(torch.int32)
    ids = torch.where(uniform(T) < case["none"], torch.full_like(ids, -1), ids)
    s["ids"] = ids[of].contiguous()
    s["s"] = empty(T, halves * R)
    s["y"] = empty(T, N)
    return s


def _act(g, kind):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    return g * 0.5 * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, kind):
    if kind == "silu":
        q = 1.0 / (1.0 + torch.exp(-g))
        return q * (1.0 + g * (1.0 - q))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _adapters_plain(s):
    """Each token's low-rank part, from the products with all adapters of the pool."""
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    n, halves, R, K = a.shape
    T, N = x.shape[0], s["N"]
    r = torch.arange(R, device=x.device)
    live = (s["ids"].long()[:, None] == torch.arange(n, device=x.device))[:, :, None, None] & (
        r < s["ranks"][:, None])[None, :, None, :]
    low = (x @ a.view(-1, K).t()).view(T, n, halves, R) * s["scale"][None, :, None, None]
    low = torch.where(live, low, torch.zeros_like(low))
    b = torch.where((r < s["ranks"][:, None])[:, None, :], b, torch.zeros_like(b)).view(n, halves, N, R)
    up = torch.matmul(low.permute(2, 0, 1, 3).reshape(halves, T, n * R),
                      b.permute(1, 0, 3, 2).reshape(halves, n * R, N).contiguous())
    return up.permute(1, 0, 2).reshape(T, halves * N)


def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "grad":
        dy = s["dy"].float()
        return {"dx": (dy @ s["w"].float()).to(torch.bfloat16), "dw": (dy.t() @ s["x"].float()).to(torch.bfloat16)}
    if op == "gated_grad":
        p, dy, F = s["p"].float(), s["dy"].float(), s["F"]
        g, u = p[:, :F], p[:, F:]
        dp = torch.cat([dy * u * _act_grad(g, s["act"]), dy * _act(g, s["act"])], 1)
        out = {"dx": (dp @ s["w"].float()).to(torch.bfloat16), "dpre": dp.to(torch.bfloat16)}
        if s["dweight"] is not None:
            out["dw"] = (dp.t() @ s["x"].float()).to(torch.bfloat16)
        return out
    v = s["x"].float() @ s["w"].float().t()
    if op == "gated":
        F = s["F"]
        out = {"h": (_act(v[:, :F], s["act"]) * v[:, F:]).to(s["h"].dtype)}
        if s["p"] is not None:
            out["pre"] = v.to(torch.bfloat16)
        return out
    v = v + _adapters_plain(s)
    if s["gated"]:
        v = _act(v[:, :s["N"]], "silu") * v[:, s["N"]:]
    return v.to(torch.bfloat16)


def _run_own(s):
    import expert_ffn_amd as lib
    op = s["op"]
    act = lib.ACT_GELU_TANH if s.get("act") == "gelu" else lib.ACT_SILU
    if op == "gated":
        lib.gated_matmul_bf16(s["x"], s["w"], act, s["h"], pre=s["p"])
        return {"h": s["h"]} if s["p"] is None else {"h": s["h"], "pre": s["p"]}
    if op == "grad":
        lib.matmul_bf16_backward(s["x"], s["w"], s["dy"], dx=s["dx"], dw=s["dweight"])
        return {"dx": s["dx"], "dw": s["dweight"]}
    if op == "gated_grad":
        lib.gated_matmul_bf16_backward(s["x"], s["w"], act, s["p"], s["dy"], s["dp"], dx=s["dx"], dw=s["dweight"])
        out = {"dx": s["dx"], "dpre": s["dp"]}
        if s["dweight"] is not None:
            out["dw"] = s["dweight"]
        return out
    lib.adapter_shrink(s["x"], s["ids"], s["a"], s["scale"], s["s"], ranks=s["ranks"])
    more = dict(s=s["s"], adapter_ids=s["ids"], b=s["b"], ranks=s["ranks"])
    if s["gated"]:
        lib.gated_matmul_bf16(s["x"], s["w"], act, s["y"], **more)
    else:
        lib.matmul_bf16(s["x"], s["w"], s["y"], **more)
    return s["y"]


def work(case):
    op, T, K = case["op"], case["T"], case["K"]
    if op == "gated":
        F = case["F"]
        return {"bytes": 2 * (T * K + 2 * F * K) + T * F * (SIZE[case["out"]] + 4 * case["pre"]), "flops": 4 * T * F * K}
    if op == "grad":
        N = case["N"]
        return {"bytes": 2 * (2 * T * K + T * N + 2 * N * K), "flops": 4 * T * N * K}
    if op == "gated_grad":
        F, both = case["F"], 2 if case["dw"] else 1
        return {"bytes": 2 * (T * K * both + 2 * F * K * both + 5 * T * F), "flops": 4 * T * F * K * both}
    N, halves = case["N"], 2 if case["gated"] else 1
    rank = case["R"] * (0.4 if case["uneven"] else 1.0)
    with_one = T * (1.0 - case["none"])
    requests = with_one if case["mix"] == "tokens" else with_one / 150
    met = case["n"] * (1.0 - (1.0 - 1.0 / case["n"]) ** requests)   # adapters of the pool that occur
    return {"bytes": 2 * (T * K + T * N + halves * N * K) + 2 * met * halves * rank * (K + N) + 4 * T,
            "flops": 2 * halves * T * N * K + 2 * halves * with_one * rank * (K + N)}


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    x, w = s["x"].to(f64), s["w"].to(f64)

    def sigma(z):
        return torch.reciprocal(1.0 + torch.exp(-z))

    def slope_and_value(g, kind):
        """act'(g), act(g): both activations are g sigma(z(g))."""
        if kind == "silu":
            z, dz = g, torch.ones_like(g)
        else:   # 0.5 (1 + tanh v) = sigma(2 v)
            c = 2.0 * math.sqrt(2.0 / math.pi)
            z, dz = c * (g + 0.044715 * g.pow(3)), c * (1.0 + 0.134145 * g.pow(2))
        q = sigma(z)
        return q + g * q * sigma(-z) * dz, g * q

    if op in ("grad", "gated_grad"):
        d = s["dy"].to(f64)
        if op == "gated_grad":
            F = case["F"]
            slope, value = slope_and_value(s["p"][:, :F].to(f64), case["act"])
            d = torch.cat([d * s["p"][:, F:].to(f64) * slope, d * value], 1)
        out = {"dx": torch.mm(d, w)}
        if case.get("dw", True):
            out["dw"] = torch.mm(d.t().contiguous(), x)
        if op == "gated_grad":
            out["dpre"] = d
        return out
    v = torch.mm(x, w.t().contiguous())
    if op == "gated":
        F = case["F"]
        out = {"h": slope_and_value(v[:, :F], case["act"])[1] * v[:, F:]}
        if case["pre"]:
            out["pre"] = v
        return out
    N = case["N"]
    for k, rank in enumerate(s["ranks"].tolist()):
        rows = (s["ids"] == k).nonzero()[:, 0]
        if not len(rows):
            continue
        for half in range(2 if case["gated"] else 1):
            low = torch.mm(x[rows], s["a"][k, half, :rank].to(f64).t().contiguous()) * s["scale"][k].to(f64)
            cols = slice(half * N, (half + 1) * N)
            v[rows, cols] += torch.mm(low, s["b"][k, cols, :rank].to(f64).t().contiguous())
    if case["gated"]:
        v = slope_and_value(v[:, :N], "silu")[1] * v[:, N:]
    return v

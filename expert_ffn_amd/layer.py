"""One MoE layer's routed expert FFN on the device: route -> permute -> expert
FFN -> combine, through the C ABI, over buffers torch allocates once.

Buffers are sized for up to T_max tokens; run() works on the first T rows.
"""
from __future__ import annotations

import torch

import expert_ffn_amd as ops

from . import (ACT_GELU_TANH, F32, GROUP_MAX, SCORE_SOFTMAX, W_BF16, W_INT8_ROW, blob_layout, combine, expert_ffn, ffn_down,
               ffn_gate_up, min_weight, permute, route_topk, router_ws_bytes, workspace_bytes)


class MoeLayer:
    def __init__(self, E, k, H, FF, fmt, T_max, device="cuda", act=ACT_GELU_TANH, renorm=1,
                 out_dtype=torch.float32, y_dtype=torch.bfloat16):
        self.E, self.k, self.H, self.FF, self.fmt, self.T_max = E, k, H, FF, fmt, T_max
        self.act, self.renorm = act, renorm
        d = torch.device(device)
        i32 = torch.int32
        self.topk_ids = torch.empty((T_max, k), dtype=i32, device=d)
        self.topk_w = torch.empty((T_max, k), dtype=torch.float32, device=d)
        self.offsets = torch.empty(E + 1, dtype=i32, device=d)
        self.sorted_route = torch.empty(T_max * k, dtype=i32, device=d)
        self.route_pos = torch.empty(T_max * k, dtype=i32, device=d)
        self.n_dropped = torch.empty(1, dtype=i32, device=d)
        self.miss_count = torch.zeros(E, dtype=i32, device=d)
        self.out_routes = torch.empty((T_max * k, H), dtype=out_dtype, device=d)
        nbytes = workspace_bytes(T_max, k, E, H, FF, fmt)
        self.ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=d)
        self.y = torch.empty((T_max, H), dtype=y_dtype, device=d)

    def views(self, T):
        k = self.k
        return dict(topk_ids=self.topk_ids[:T], topk_w=self.topk_w[:T], offsets=self.offsets,
                    sorted_route=self.sorted_route[:T * k], route_pos=self.route_pos[:T * k],
                    n_dropped=self.n_dropped, out_routes=self.out_routes[:T * k], y=self.y[:T])

    def route(self, logits, stream=None):
        T = logits.shape[0]
        route_topk(logits, self.k, self.topk_ids[:T], self.topk_w[:T], self.renorm, stream)
        self.group(T, stream)

    def select(self, logits, share, stream=None):
        """Top-k, then min_weight partial routing at `share` in place; leaves
        in miss_count the kept routes per non-resident expert (the experts to
        fill before group())."""
        T = logits.shape[0]
        route_topk(logits, self.k, self.topk_ids[:T], self.topk_w[:T], self.renorm, stream)
        min_weight(self.topk_ids[:T], self.topk_w[:T], self.E, self._slot_of, share, self.topk_ids[:T],
                   self.topk_w[:T], self.miss_count, stream)

    def group(self, T, stream=None):
        """Permute the current top-k routes against the bound slot table."""
        permute(self.topk_ids[:T], self.E, self._slot_of, self.offsets, self.sorted_route[:T * self.k],
                self.route_pos[:T * self.k], self.n_dropped, stream)

    def ffn(self, x, stream=None):
        T = x.shape[0]
        expert_ffn(self._pool, self._slot_bytes, self._slot_of, self.E, self.H, self.FF, self.fmt,
                   self.act, x, self.k, self.offsets, self.sorted_route[:T * self.k],
                   self.out_routes[:T * self.k], self.ws, stream)

    def gate_up(self, x, stream=None):
        ffn_gate_up(self._pool, self._slot_bytes, self._slot_of, self.E, self.H, self.FF, self.fmt,
                    self.act, x, self.k, self.offsets, self.sorted_route[:x.shape[0] * self.k], self.ws,
                    stream)

    def down(self, T, stream=None):
        ffn_down(self._pool, self._slot_bytes, self._slot_of, self.E, self.H, self.FF, self.fmt, T,
                 self.k, self.offsets, self.sorted_route[:T * self.k], self.out_routes[:T * self.k],
                 self.ws, stream)

    def combine(self, T, stream=None):
        combine(self.out_routes[:T * self.k], self.topk_w[:T], self.route_pos[:T * self.k],
                self.y[:T], stream)

    def bind(self, pool, slot_bytes, slot_of):
        """Select the layer's experts: a slot pool, its slot size and expert -> slot table."""
        self._pool, self._slot_bytes, self._slot_of = pool, int(slot_bytes), slot_of
        return self

    def run(self, logits, x, stream=None):
        """The whole layer for T = logits.shape[0] tokens; returns the y view."""
        T = logits.shape[0]
        self.route(logits, stream)
        self.ffn(x, stream)
        self.combine(T, stream)
        return self.y[:T]


class DenseExpert:
    """A dense (shared) expert beside the routed ones, in 8-bit integers: an int8 blob (pack_expert with
    W_INT8_ROW) whose codes the 8-bit products read in place."""

    def __init__(self, blob, H, FF, act=ACT_GELU_TANH):
        o13, s13, o2, s2, size = blob_layout(W_INT8_ROW, H, FF)
        if blob.dtype != torch.uint8 or not blob.is_contiguous() or blob.numel() < size:
            raise ValueError(f"blob must be {size} contiguous bytes")
        b = blob.view(-1)
        self.H, self.FF, self.act, self.blob = H, FF, act, blob
        self.w13 = b[o13:o13 + 2 * FF * H].view(torch.int8).view(2 * FF, H)
        self.s13 = b[s13:s13 + 8 * FF].view(torch.float32)
        self.w2 = b[o2:o2 + H * FF].view(torch.int8).view(H, FF)
        self.s2 = b[s2:s2 + 4 * H].view(torch.float32)


class Adapters:
    """Low-rank adapters of a DenseExpertBf16 for many requests at once: a pool of n slots of at most R ranks.
    A request's tokens carry its slot's number; a slot that is not loaded has rank 0 and adds nothing."""

    def __init__(self, n, R, H, FF, device="cuda"):
        if n < 1 or R < 8 or R > 1024 or R % 8:
            raise ValueError(f"n={n} is not positive, or R={R} not a multiple of 8 in [8, 1024]")
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.n, self.R, self.H, self.FF = n, R, H, FF
        self.a13, self.b13 = torch.zeros((n, 2, R, H), **bf16), torch.zeros((n, 2 * FF, R), **bf16)
        self.a2, self.b2 = torch.zeros((n, R, FF), **bf16), torch.zeros((n, H, R), **bf16)
        self.scale = torch.ones(n, dtype=torch.float32, device=device)
        self.ranks = torch.zeros(n, dtype=torch.int32, device=device)

    @torch.no_grad()   # the pools keep no graph of parameters that are loaded
    def load(self, slot, a13, b13, a2, b2, scale=1.0):
        """a13 [2, r, H] (gate, up), b13 [2FF, r], a2 [r, FF], b2 [H, r] into a slot, on the current stream."""
        r = a2.shape[0]
        if not 0 <= slot < self.n:
            raise ValueError(f"slot {slot} outside [0, {self.n})")
        shapes = [tuple(t.shape) for t in (a13, b13, a2, b2)]
        if r > self.R or shapes != [(2, r, self.H), (2 * self.FF, r), (r, self.FF), (self.H, r)]:
            raise ValueError(f"adapter shapes {shapes} do not fit slots of rank {self.R}, H={self.H}, FF={self.FF}")
        self.a13[slot, :, :r] = a13
        self.b13[slot, :, :r] = b13
        self.a2[slot, :r] = a2
        self.b2[slot, :, :r] = b2
        self.scale[slot] = scale
        self.ranks[slot] = r


class DenseExpertBf16:
    """A dense (shared) expert beside the routed ones, in bf16: a bf16 blob (pack_expert with W_BF16) read in place,
    with the adapters of the tokens' requests (an Adapters, or None) and the backward pass of the expert."""

    def __init__(self, blob, H, FF, act=ACT_GELU_TANH, adapters=None):
        o13, _, o2, _, size = blob_layout(W_BF16, H, FF)
        if blob.dtype != torch.uint8 or not blob.is_contiguous() or blob.numel() < size:
            raise ValueError(f"blob must be {size} contiguous bytes")
        if adapters is not None and (adapters.H, adapters.FF) != (H, FF):
            raise ValueError(f"the adapters have H={adapters.H}, FF={adapters.FF}, the expert {H}, {FF}")
        b = blob.view(-1)
        self.H, self.FF, self.act, self.blob, self.adapters = H, FF, act, blob, adapters
        self.w13 = b[o13:o13 + 4 * FF * H].view(torch.bfloat16).view(2 * FF, H)
        self.w2 = b[o2:o2 + 2 * H * FF].view(torch.bfloat16).view(H, FF)

    def run(self, x, hid, y, pre=None, low=None, adapter_ids=None, stream=None):
        """hid [T, FF] = act(gate) up of x [T, H], y [T, H] = hid . w2.  pre [T, 2FF] takes the sums of gate and up for
        backward(); adapter_ids [T] the tokens' slots, with low [T, 2R] for the adapters' first products.  Not both:
        the backward pass has no adapters."""
        more, more2 = {}, {}
        if adapter_ids is not None:
            a = self.adapters
            if a is None:
                raise ValueError("adapter_ids are given, but the expert has no adapters")
            if low is None:
                raise ValueError("adapter_ids need low")
            if pre is not None:
                raise ValueError("pre goes with a pass without adapters: backward() has none of their terms")
            low2 = low[:, :a.R]   # reused behind gate and up
            ops.adapter_shrink(x, adapter_ids, a.a13, a.scale, low, ranks=a.ranks, stream=stream)
            more = dict(s=low, adapter_ids=adapter_ids, b=a.b13, ranks=a.ranks)
            more2 = dict(s=low2, adapter_ids=adapter_ids, b=a.b2, ranks=a.ranks)
        ops.gated_matmul_bf16(x, self.w13, self.act, hid, pre=pre, stream=stream, **more)
        if more2:
            ops.adapter_shrink(hid, adapter_ids, a.a2, a.scale, low2, ranks=a.ranks, stream=stream)
        ops.matmul_bf16(hid, self.w2, y, stream=stream, **more2)
        return y

    def backward(self, x, pre, hid, dy, dhid, dpre, dx=None, dw13=None, dw2=None, stream=None):
        """Gradients of run() without adapters, from what it read and stored (pre and hid of one call without adapter_ids)
        and dy [T, H]: dhid [T, FF] and dpre [T, 2FF] (may be pre) on the way, dx [T, H], dw13 and dw2 where they are
        wanted.  dhid and dpre are bf16, so dx and dw13 carry their rounding in fp32 too."""
        ops.matmul_bf16_backward(hid, self.w2, dy, dx=dhid, dw=dw2, stream=stream)
        ops.gated_matmul_bf16_backward(x, self.w13, self.act, pre, dhid, dpre, dx=dx, dw=dw13, stream=stream)


class MoeBlock:
    """The MoE half of a transformer block around a MoeLayer, over buffers torch allocates once:

        x      = norm(h; w_in)              bf16, and 8-bit codes for a dense expert in 8 bits
        routes = scored top-k of x . w_router^T, grouped by expert
        h_out  = res_scale h + block_scale gate norm(combine(routes) + dense(x); w_post)

    run() returns h_out [T, H] and, with w_next, the next block's normed rows.  h is fp32 or bf16; h_out
    may be h.  w_post, gate, bias, dense and w_next may be None.  The buffers hold up to the layer's T_max
    tokens and are reused by the next run: calls on one block are ordered by the caller.

    dense is a DenseExpert (8-bit weights and activations) or a DenseExpertBf16, whose adapters run() takes by
    the tokens' slots.

    One norm (w_in) feeds the router, the routed and the dense experts, and one (w_post) covers the sum of
    what they give.  A block that norms these apart calls norm_in, router_score_topk, the layer's steps and
    norm_out itself (y takes the rows of any dense expert)."""

    def __init__(self, layer, w_in, w_router, w_post=None, eps=1e-6, w_offset=0.0, dense=None, gate=None,
                 block_scale=1.0, res_scale=1.0, w_next=None, score=SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1,
                 group_rank=GROUP_MAX, route_scale=1.0):
        T, H, d = layer.T_max, layer.H, layer.y.device
        if dense is not None and dense.H != H:
            raise ValueError(f"the dense expert has H={dense.H}, the layer {H}")
        self.layer, self.dense, self.gate, self.eps, self.w_offset = layer, dense, gate, eps, w_offset
        self.w_in, self.w_router, self.w_post, self.w_next = w_in, w_router, w_post, w_next
        self.block_scale, self.res_scale = block_scale, res_scale
        self.routing = dict(score=score, bias=bias, n_group=n_group, topk_group=topk_group, group_rank=group_rank,
                            renorm=layer.renorm, scale=route_scale)
        bf16, f32 = torch.bfloat16, torch.float32
        self.x = torch.empty((T, H), dtype=bf16, device=d)
        self.logits = torch.empty((T, layer.E), dtype=f32, device=d)
        # enough for fewer tokens too: their slices of H are as many or fewer
        self.router_ws = torch.empty(max(router_ws_bytes(T, H, layer.E), 256), dtype=torch.uint8, device=d)
        self.x_next = torch.empty((T, H), dtype=bf16, device=d) if w_next is not None else None
        self.codes = dense is not None and not isinstance(dense, DenseExpertBf16)
        if dense is not None:
            self.hid = torch.empty((T, dense.FF), dtype=bf16, device=d)
            self.yd = torch.empty((T, H), dtype=bf16, device=d)
        if self.codes:
            self.xq = torch.empty((T, H), dtype=torch.int8, device=d)
            self.hq = torch.empty((T, dense.FF), dtype=torch.int8, device=d)
            self.xs, self.hs = (torch.empty(T, dtype=f32, device=d) for _ in range(2))
        a = dense.adapters if isinstance(dense, DenseExpertBf16) else None
        self.low = torch.empty((T, 2 * a.R), dtype=bf16, device=d) if a is not None else None

    def _check_ids(self, adapter_ids):
        if adapter_ids is not None and self.low is None:
            raise ValueError("adapter_ids are given, but the dense expert has no adapters")

    def run_dense(self, T, stream=None, adapter_ids=None):
        """The dense expert on the rows (or their codes) of the last norm: its rows in yd."""
        self._check_ids(adapter_ids)
        e = self.dense
        if not self.codes:
            low = self.low[:T] if self.low is not None else None
            return e.run(self.x[:T], self.hid[:T], self.yd[:T], low=low, adapter_ids=adapter_ids, stream=stream)
        ops.gated_matmul_i8(self.xq[:T], self.xs[:T], e.w13, e.s13, e.act, self.hid[:T], stream)
        ops.quantize_tokens(self.hid[:T], self.hq[:T], self.hs[:T], stream)
        ops.matmul_i8(self.hq[:T], self.hs[:T], e.w2, e.s2, self.yd[:T], stream=stream)
        return self.yd[:T]

    def run(self, h, h_out, stream=None, adapter_ids=None):
        """adapter_ids: int32 [T], the slots of the tokens' adapters in the dense expert's pool (outside it: none)."""
        self._check_ids(adapter_ids)
        if h.shape[0] > self.layer.T_max:
            raise ValueError(f"T={h.shape[0]} exceeds the layer's T_max={self.layer.T_max}")
        if h.shape[0] == 0:
            return h_out, self.x_next[:0] if self.x_next is not None else None
        with torch.cuda.device(self.x.device):   # the layer's calls go to the current device
            return self._run(h, h_out, stream, adapter_ids)

    def _run(self, h, h_out, stream, adapter_ids):
        T, L = h.shape[0], self.layer
        codes = dict(xq=self.xq[:T], xq_scale=self.xs[:T]) if self.codes else {}
        ops.norm_in(h, self.w_in, self.eps, x=self.x[:T], w_offset=self.w_offset, stream=stream, **codes)
        ops.router_score_topk(self.x[:T], self.w_router, L.k, self.logits[:T], self.router_ws, L.topk_ids[:T],
                              L.topk_w[:T], stream=stream, **self.routing)
        L.group(T, stream)
        L.ffn(self.x[:T], stream)
        y = self.run_dense(T, stream, adapter_ids) if self.dense is not None else None
        gate = self.gate[:T] if self.gate is not None and self.gate.dim() == 2 and self.gate.shape[0] > 1 else self.gate
        nxt = self.x_next[:T] if self.x_next is not None else None
        ops.norm_out(h, h_out, self.w_post, self.eps, out_routes=L.out_routes[:T * L.k], topk_w=L.topk_w[:T],
                     route_pos=L.route_pos[:T * L.k], y=y, gate=gate, block_scale=self.block_scale,
                     res_scale=self.res_scale, w_next=self.w_next, x=nxt, w_offset=self.w_offset, stream=stream)
        return h_out, nxt


__all__ = ["MoeLayer", "MoeBlock", "DenseExpert", "DenseExpertBf16", "Adapters", "F32"]

"""Python binding of libexpert_ffn.so (the C ABI in include/expert_ffn.h).

Argument marshalling only: every function passes torch tensors' device
pointers, sizes and torch's current HIP stream to the C entry point of the same
name and raises MoeError on a non-OK status.  There is no fallback: without the
built library, importing the first entry point raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libexpert_ffn.so")

F32, BF16 = 0, 1
W_BF16, W_INT8_ROW, W_INT4_G64 = 0, 1, 2
ACT_GELU_TANH, ACT_SILU = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
FMT_NAMES = {"bf16": W_BF16, "int8": W_INT8_ROW, "int4": W_INT4_G64}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"status {status}: {message}")
        self.status = status


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_expert_bytes.argtypes = [i32, i32, i32]
        L.moe_expert_bytes.restype = u64
        L.moe_blob_layout.argtypes = [i32, i32, i32, P]
        L.moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
        L.moe_workspace_bytes.restype = sz
        L.moe_route_topk.argtypes = [P, i32, i32, i32, i32, P, P, P]
        L.moe_permute.argtypes = [P, i32, i32, i32, P, P, P, P, P, P]
        L.moe_route_permute.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P, P, P, P]
        ffn = [P, u64, P, i32, i32, i32, i32, i32, P, i32, i32, i32, P, P, P, i32, P, sz, P]
        for name in ("moe_expert_ffn", "moe_ffn_gate_up", "moe_ffn_down"):
            getattr(L, name).argtypes = ffn
        L.moe_expert_ffn_noalloc.argtypes = ffn[:16] + [P]
        L.moe_combine.argtypes = [P, i32, P, P, i32, i32, i32, P, i32, P]
        L.moe_quantize.argtypes = [i32, P, i32, i32, P, P, P]
        L.moe_pack_expert.argtypes = [i32, P, P, i32, i32, P, P]
        L.moe_router_ws_bytes.argtypes = [i32, i32, i32]
        L.moe_router_ws_bytes.restype = sz
        L.moe_router_topk.argtypes = [P, i32, i32, i32, P, i32, i32, i32, P, P, sz, P, P, P]
        L.moe_residency_refresh.argtypes = [P, ctypes.c_int64, i32, i32, i32, P, P, P, P, P, P, P, P]
        L.moe_refresh_due.argtypes = [i32, ctypes.c_int64, i32, i32]
        L.moe_refresh_due.restype = i32
        L.moe_budget_from_memory.argtypes = [u64, u64, u64, i32, i32, i32]
        L.moe_budget_from_memory.restype = i32
        L.moe_min_weight.argtypes = [P, P, i32, i32, i32, P, ctypes.c_float, P, P, P, P]
        L.moe_fill_slot.argtypes = [i32, P, i32, i32, i32, P, P, P]
        L.moe_fill_slots.argtypes = [i32, i32, P, i32, i32, P, P, P]
        L.moe_verify_slot.argtypes = [i32, P, i32, i32, P, P, P]
        L.moe_slot_admit.argtypes = [P, i32, P, i32, i32]
        f32, i64 = ctypes.c_float, ctypes.c_int64
        L.moe_route_score_topk.argtypes = [P, i32, i64, P, i32, i32, i32, i32, i32, i32, i32, i32, f32, P, P, P]
        L.moe_router_score_topk.argtypes = [P, i32, i32, i32, P, i32, i32, P, i32, i32, i32, i32, i32, f32, P, P, sz, P, P, P]
        L.moe_norm_in.argtypes = [P, i32, i64, i32, i32, P, i32, f32, f32, P, i32, i64, P, i64, P, P]
        L.moe_norm_out.argtypes = [P, i32, P, P, i32, P, i32, i64, i32, i32, P, i32, f32, f32, P, i32, i64, i64, f32, f32,
                                   P, i32, i64, P, i64, i32, P, P, i32, i64, P, i64, P, P]
        L.moe_quantize_tokens.argtypes = [P, i32, i64, i32, i32, P, i64, P, P]
        L.moe_matmul_i8.argtypes = [P, i64, P, P, i64, P, P, i32, i32, i32, P, i32, i64, P]
        L.moe_gated_matmul_i8.argtypes = [P, i64, P, P, i64, P, i32, i32, i32, i32, P, i32, i64, P]
        for name in ("moe_route_score_topk", "moe_router_score_topk", "moe_norm_in", "moe_norm_out", "moe_quantize_tokens", "moe_matmul_i8",
                     "moe_gated_matmul_i8"):
            getattr(L, name).restype = ctypes.c_int
        for name in ("moe_blob_layout", "moe_route_topk", "moe_permute", "moe_route_permute", "moe_expert_ffn",
                     "moe_ffn_gate_up", "moe_ffn_down", "moe_expert_ffn_noalloc", "moe_combine", "moe_quantize",
                     "moe_pack_expert", "moe_router_topk", "moe_residency_refresh", "moe_min_weight", "moe_fill_slot", "moe_fill_slots", "moe_verify_slot",
                     "moe_slot_admit"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        raise MoeError(status, lib().moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------ host queries --
def expert_bytes(fmt: int, H: int, FF: int) -> int:
    return int(lib().moe_expert_bytes(fmt, H, FF))


def blob_layout(fmt: int, H: int, FF: int):
    off = (ctypes.c_uint64 * 5)()
    _check(lib().moe_blob_layout(fmt, H, FF, off))
    return [int(v) for v in off]


def workspace_bytes(T: int, k: int, E: int, H: int, FF: int, fmt: int) -> int:
    return int(lib().moe_workspace_bytes(T, k, E, H, FF, fmt))


# ------------------------------------------------------------- the steps --
def route_topk(logits, k: int, topk_ids, topk_w, renorm: int = 1, stream=None):
    T, E = logits.shape
    _check(lib().moe_route_topk(_ptr(logits), T, E, k, renorm, _ptr(topk_ids), _ptr(topk_w),
                                _stream(stream)))


def permute(topk_ids, E: int, slot_of, expert_offsets, sorted_route, route_pos, n_dropped,
            stream=None):
    T, k = topk_ids.shape
    _check(lib().moe_permute(_ptr(topk_ids), T, k, E, _ptr(slot_of), _ptr(expert_offsets),
                             _ptr(sorted_route), _ptr(route_pos), _ptr(n_dropped), _stream(stream)))


def route_permute(logits, k: int, slot_of, topk_ids, topk_w, expert_offsets, sorted_route, route_pos,
                  n_dropped, renorm: int = 1, stream=None):
    T, E = logits.shape
    _check(lib().moe_route_permute(_ptr(logits), T, E, k, renorm, _ptr(slot_of), _ptr(topk_ids), _ptr(topk_w),
                                   _ptr(expert_offsets), _ptr(sorted_route), _ptr(route_pos), _ptr(n_dropped),
                                   _stream(stream)))


def _ffn(name, pool, slot_bytes, slot_of, E, H, FF, fmt, act, x, T, k, expert_offsets,
         sorted_route, out_routes, ws, stream):
    x_dt = _dt(x) if x is not None else BF16
    o_dt = _dt(out_routes) if out_routes is not None else F32
    _check(getattr(lib(), name)(_ptr(pool), slot_bytes, _ptr(slot_of), E, H, FF, fmt, act, _ptr(x),
                                x_dt, T, k, _ptr(expert_offsets), _ptr(sorted_route),
                                _ptr(out_routes), o_dt, _ptr(ws), ws.numel() * ws.element_size(),
                                _stream(stream)))


def expert_ffn(pool, slot_bytes, slot_of, E, H, FF, fmt, act, x, k, expert_offsets, sorted_route,
               out_routes, ws, stream=None):
    _ffn("moe_expert_ffn", pool, slot_bytes, slot_of, E, H, FF, fmt, act, x, x.shape[0], k,
         expert_offsets, sorted_route, out_routes, ws, stream)


def expert_ffn_noalloc(pool, slot_bytes, slot_of, E, H, FF, fmt, act, x, k, expert_offsets, sorted_route,
                       out_routes, stream=None):
    """moe_expert_ffn_noalloc: the library's static scratch array is the workspace."""
    _check(lib().moe_expert_ffn_noalloc(_ptr(pool), slot_bytes, _ptr(slot_of), E, H, FF, fmt, act, _ptr(x),
                                        _dt(x), x.shape[0], k, _ptr(expert_offsets), _ptr(sorted_route),
                                        _ptr(out_routes), _dt(out_routes), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20


def ffn_gate_up(pool, slot_bytes, slot_of, E, H, FF, fmt, act, x, k, expert_offsets,
                sorted_route, ws, stream=None):
    _ffn("moe_ffn_gate_up", pool, slot_bytes, slot_of, E, H, FF, fmt, act, x, x.shape[0], k,
         expert_offsets, sorted_route, None, ws, stream)


def ffn_down(pool, slot_bytes, slot_of, E, H, FF, fmt, T, k, expert_offsets, sorted_route,
             out_routes, ws, stream=None):
    _ffn("moe_ffn_down", pool, slot_bytes, slot_of, E, H, FF, fmt, ACT_GELU_TANH, None, T, k,
         expert_offsets, sorted_route, out_routes, ws, stream)


def combine(out_routes, topk_w, route_pos, y, stream=None):
    T, H = y.shape
    k = topk_w.numel() // T if T else 1
    _check(lib().moe_combine(_ptr(out_routes), _dt(out_routes), _ptr(topk_w), _ptr(route_pos), T, k,
                             H, _ptr(y), _dt(y), _stream(stream)))


def quantize(fmt: int, w_bf16, q, scales, stream=None):
    N, K = w_bf16.shape
    _check(lib().moe_quantize(fmt, _ptr(w_bf16), N, K, _ptr(q), _ptr(scales), _stream(stream)))


def pack_expert(fmt: int, w13_bf16, w2_bf16, blob, stream=None):
    H = w13_bf16.shape[1]
    FF = w2_bf16.shape[1]
    _check(lib().moe_pack_expert(fmt, _ptr(w13_bf16), _ptr(w2_bf16), H, FF, _ptr(blob),
                                 _stream(stream)))


def fill_slot(fmt: int, src, H: int, FF: int, slot, staging=None, stream=None, direct=False):
    """Canonical blob src (host: one copy into staging, then the unpack kernel,
    or with direct=True the kernel reading the pinned blob itself; device: the
    kernel alone) -> slot, byte for byte the packed blob."""
    on_host = 0 if src.is_cuda else (2 if direct else 1)
    _check(lib().moe_fill_slot(fmt, _ptr(src), on_host, H, FF, _ptr(staging), _ptr(slot), _stream(stream)))


def fill_slots(fmt: int, srcs, H: int, FF: int, slots, staging, stream=None):
    """Canonical blobs srcs (host tensors) -> slots (device tensors): the
    copies back to back into staging, then one unpack kernel for all."""
    n = len(srcs)
    assert len(slots) == n
    src_arr = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in srcs])
    dst_arr = (ctypes.c_void_p * max(n, 1))(*[t.data_ptr() for t in slots])
    _check(lib().moe_fill_slots(fmt, n, src_arr, H, FF, _ptr(staging), dst_arr, _stream(stream)))


def verify_slot(fmt: int, src, H: int, FF: int, slot, mismatches, stream=None):
    """mismatches[0] <- 16-byte chunks of slot that differ from the fill of src."""
    _check(lib().moe_verify_slot(fmt, _ptr(src), H, FF, _ptr(slot), _ptr(mismatches), _stream(stream)))


def slot_admit(slot_of, owner, expert: int) -> int:
    """Host int32 tables slot_of [E], owner [S]: expert's slot, claiming the
    lowest free one if it is not resident; raises when none is free."""
    import torch
    assert slot_of.dtype == torch.int32 and owner.dtype == torch.int32
    assert not slot_of.is_cuda and not owner.is_cuda and slot_of.is_contiguous() and owner.is_contiguous()
    j = lib().moe_slot_admit(_ptr(slot_of), slot_of.numel(), _ptr(owner), owner.numel(), expert)
    if j < 0:
        raise MoeError(1, lib().moe_last_error().decode())
    return j


def min_weight(ids, w, E: int, slot_of, share: float, ids_out, w_out, miss_count, stream=None):
    """min_weight partial routing of topk ids/w [T, k] (outputs may alias them)."""
    T, k = ids.shape
    _check(lib().moe_min_weight(_ptr(ids), _ptr(w), T, k, E, _ptr(slot_of), ctypes.c_float(share), _ptr(ids_out),
                                _ptr(w_out), _ptr(miss_count), _stream(stream)))


def router_ws_bytes(T: int, H: int, E: int) -> int:
    """Bytes of the workspace router_topk needs for T tokens."""
    return int(lib().moe_router_ws_bytes(T, H, E))


def router_topk(x, w_router, k: int, logits, ws, ids, w, renorm: int = 1, stream=None):
    """fp32 router GEMV of x [T, H] with w_router [E, H], then the top-k (two launches)."""
    T, H = x.shape
    E = w_router.shape[0]
    _check(lib().moe_router_topk(_ptr(x), _dt(x), T, H, _ptr(w_router), E, k, renorm, _ptr(logits), _ptr(ws),
                                 ws.numel() * ws.element_size(), _ptr(ids), _ptr(w), _stream(stream)))


def residency_refresh(ids, E: int, budget: int, n_slots: int, slot_of, hits, target, promote, promote_slot, demote,
                      counts, stream=None):
    """Hit counts, top-budget target and paired promote/demote; slot_of is rewritten in place."""
    _check(lib().moe_residency_refresh(_ptr(ids), ids.numel(), E, budget, n_slots, _ptr(slot_of), _ptr(hits),
                                       _ptr(target), _ptr(promote), _ptr(promote_slot), _ptr(demote), _ptr(counts),
                                       _stream(stream)))


def refresh_due(every: int, step: int, prefill_block: bool, offload: bool) -> bool:
    return bool(lib().moe_refresh_due(every, step, int(prefill_block), int(offload)))


def budget_from_memory(free_bytes: int, reserve_bytes: int, expert_bytes: int, layers: int, max_per_layer: int,
                       E: int) -> int:
    return int(lib().moe_budget_from_memory(free_bytes, reserve_bytes, expert_bytes, layers, max_per_layer, E))


# --------------------------------------------- around the expert FFN --
# These calls check shapes, types and devices here, take rows at any stride
# (elements of a row contiguous), and run on the tensors' device: on its
# current stream when none is given.
_DT = None
_raw_stream = _device = None


def _setup():
    """torch's type codes and its queries of the current device and its raw stream (torch is imported on
    first use only).  The public current_stream() and current_device() cost 2 us of a call that takes 6."""
    global _DT, _raw_stream, _device
    import torch
    lib()
    _raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _DT = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: "int8", torch.int32: "int32"}


def _type_error(name, t):
    return TypeError(f"unsupported dtype {t.dtype} of {name}")


def _where_error(name, t, dev):
    return ValueError(f"{name} is on {t.device}, expected GPU {dev}")


def _mat(name, t, rows, cols, dev, kind=None):
    """(pointer, dtype code, row stride) of t [rows, cols] on GPU dev; kind None: fp32 or bf16, else that type."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.get_device() != dev:
        raise _where_error(name, t, dev)
    code = _DT.get(t.dtype)
    if (code != kind) if kind is not None else (code != F32 and code != BF16):
        raise _type_error(name, t)
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"the elements of a row of {name} are not contiguous")
    return t.data_ptr(), code, (s0 if rows > 1 else cols)


def _first(name, t, kind=None):
    """(GPU, rows, columns, pointer, dtype code, row stride) of the matrix whose shape the others follow."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} is on {t.device}: a GPU is needed")
    if t.dim() != 2:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected 2")
    if _DT is None:
        _setup()
    rows, cols = t.shape
    return (dev, rows, cols) + _mat(name, t, rows, cols, dev, kind)


def _vec(name, t, n, dev, kind=None):
    """(pointer, dtype code) of the n contiguous elements of t on GPU dev (n in all, whatever the shape)."""
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    if t.get_device() != dev:
        raise _where_error(name, t, dev)
    code = _DT.get(t.dtype)
    if (code != kind) if kind is not None else (code != F32 and code != BF16):
        raise _type_error(name, t)
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return t.data_ptr(), code


def _on(dev, stream, fn, *args):
    """Call fn on GPU dev's current stream (or `stream`, one of that GPU's), with dev current."""
    if stream is None:
        s = _raw_stream(dev)
    else:
        if stream.device_index != dev:
            raise ValueError(f"the stream belongs to GPU {stream.device_index}, the tensors are on GPU {dev}")
        s = stream.cuda_stream
    if _device() == dev:
        rc = fn(*args, s)
    else:
        import torch
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        _check(rc)


def route_score_topk(logits, k: int, topk_ids, topk_w, score: int = SCORE_SOFTMAX, bias=None, n_group: int = 1,
                     topk_group: int = 1, group_rank: int = GROUP_MAX, renorm: int = 1, scale: float = 1.0,
                     stream=None):
    """Top-k of softmax or sigmoid scores of logits [T, E] plus a bias [E] that counts for the choice
    only, inside the topk_group best of n_group expert groups; ids int32 and weights fp32 [T, k]."""
    dev, T, E, lp, ldt, ld = _first("logits", logits)
    bp = None if bias is None else _vec("bias", bias, E, dev, F32)[0]
    ip = _vec("topk_ids", topk_ids, T * k, dev, "int32")[0]
    wp = _vec("topk_w", topk_w, T * k, dev, F32)[0]
    _on(dev, stream, _lib.moe_route_score_topk, lp, ldt, ld, bp, T, E, k, score, n_group, topk_group, group_rank, renorm,
        scale, ip, wp)


def router_score_topk(x, w_router, k: int, logits, ws, topk_ids, topk_w, score: int = SCORE_SOFTMAX, bias=None,
                      n_group: int = 1, topk_group: int = 1, group_rank: int = GROUP_MAX, renorm: int = 1,
                      scale: float = 1.0, stream=None):
    """fp32 router product of x [T, H] with w_router [E, H] (logits [T, E] out, ws as for router_topk), then
    route_score_topk on the logits."""
    dev, T, H, xp, xdt, ldx = _first("x", x)
    if ldx != H and T > 1:
        raise ValueError("x is not contiguous")
    E = w_router.shape[0]
    wp = _vec("w_router", w_router, E * H, dev, F32)[0]
    lp = _vec("logits", logits, T * E, dev, F32)[0]
    bp = None if bias is None else _vec("bias", bias, E, dev, F32)[0]
    ip = _vec("topk_ids", topk_ids, T * k, dev, "int32")[0]
    op = _vec("topk_w", topk_w, T * k, dev, F32)[0]
    if ws.get_device() != dev:
        raise _where_error("ws", ws, dev)
    if not ws.is_contiguous():
        raise ValueError("ws is not contiguous")
    _on(dev, stream, _lib.moe_router_score_topk, xp, xdt, T, H, wp, E, k, bp, score, n_group, topk_group, group_rank, renorm,
        scale, lp, ws.data_ptr(), ws.numel() * ws.element_size(), ip, op)


def _norm_outputs(T, H, dev, x, xq, xq_scale):
    xp, xdt, ldx = (None, F32, 0) if x is None else _mat("x", x, T, H, dev)
    if (xq is None) != (xq_scale is None):
        raise ValueError("xq and xq_scale go together")
    if xq is None:
        return xp, xdt, ldx, None, 0, None
    qp, _, ldq = _mat("xq", xq, T, H, dev, "int8")
    return xp, xdt, ldx, qp, ldq, _vec("xq_scale", xq_scale, T, dev, F32)[0]


def norm_in(h, w, eps: float, x=None, xq=None, xq_scale=None, w_offset: float = 0.0, stream=None):
    """RMS norm of the rows of h [T, H] with weight w_offset + w [H] (w None: 1), into x (fp32 or bf16),
    as int8 codes xq with one fp32 scale per row (xq_scale [T]), or both."""
    dev, T, H, hp, hdt, ldh = _first("h", h)
    wp, wdt = (None, F32) if w is None else _vec("w", w, H, dev)
    _on(dev, stream, _lib.moe_norm_in, hp, hdt, ldh, T, H, wp, wdt, w_offset, eps,
        *_norm_outputs(T, H, dev, x, xq, xq_scale))


def quantize_tokens(x, xq, xq_scale, stream=None):
    """int8 codes and the scale of each row of x [T, K]: codes rint(x / s), s = max |x| / 127."""
    dev, T, K, xp, xdt, ldx = _first("x", x)
    qp, _, ldq = _mat("xq", xq, T, K, dev, "int8")
    _on(dev, stream, _lib.moe_quantize_tokens, xp, xdt, ldx, T, K, qp, ldq, _vec("xq_scale", xq_scale, T, dev, F32)[0])


def norm_out(h, h_out, w_post, eps: float, out_routes=None, topk_w=None, route_pos=None, y=None, gate=None,
             block_scale: float = 1.0, res_scale: float = 1.0, w_next=None, x=None, xq=None, xq_scale=None,
             w_offset: float = 0.0, stream=None):
    """End of a block: h_out = res_scale * h + block_scale * gate * norm(b; w_post), where b is the weighted
    combine of out_routes (topk_w, route_pos [T, k] as for combine) plus y [T, H]; then, when x or xq is
    given, the next block's norm of h_out (w_next) into them.  w_post None: b is not normed.  gate
    broadcasts to [T, H].  h_out may be h."""
    dev, T, H, hp, hdt, ldh = _first("h", h)
    op, _, ldo = _mat("h_out", h_out, T, H, dev, hdt)
    rp = wp = pp = None
    rdt, k = F32, 0
    if out_routes is not None:
        if topk_w is None or route_pos is None:
            raise ValueError("out_routes needs topk_w and route_pos")
        R = route_pos.numel()
        k = R // T if T else 0
        if k * T != R:
            raise ValueError(f"route_pos has {R} elements, not a multiple of T={T}")
        if not out_routes.is_contiguous():
            raise ValueError("out_routes is not contiguous")
        rp, rdt, _ = _mat("out_routes", out_routes, R, H, dev)
        wp = _vec("topk_w", topk_w, R, dev, F32)[0]
        pp = _vec("route_pos", route_pos, R, dev, "int32")[0]
    yp, ydt, ldy = (None, F32, 0) if y is None else _mat("y", y, T, H, dev)
    pw, wdt = (None, F32) if w_post is None else _vec("w_post", w_post, H, dev)
    nw = None
    if w_next is not None:
        nw, ndt = _vec("w_next", w_next, H, dev)
        if w_post is not None and ndt != wdt:
            raise TypeError("w_post and w_next have different dtypes")
        wdt = ndt
    gp, gdt, gst, gsh = None, F32, 0, 0
    if gate is not None:
        # broadcast by hand: gate.expand() alone takes 2 us
        nd = gate.dim()
        gr, gc = (1,) * (2 - nd) + tuple(gate.shape) if nd <= 2 else (0, 0)
        if (gr != 1 and gr != T) or (gc != 1 and gc != H):
            raise ValueError(f"gate has shape {tuple(gate.shape)}, which does not broadcast to {(T, H)}")
        if gate.get_device() != dev:
            raise _where_error("gate", gate, dev)
        gdt = _DT.get(gate.dtype)
        if gdt != F32 and gdt != BF16:
            raise _type_error("gate", gate)
        st = gate.stride()
        if gr > 1:
            gst = st[0]
        if gc > 1:
            gsh = st[-1]
        gp = gate.data_ptr()
    outs = _norm_outputs(T, H, dev, x, xq, xq_scale)
    nxt = int(x is not None or xq is not None)
    if w_next is not None and not nxt:
        raise ValueError("w_next is given, but neither x nor xq to write the next norm into")
    _on(dev, stream, _lib.moe_norm_out, rp, rdt, wp, pp, k, yp, ydt, ldy, T, H, pw, wdt, w_offset, eps, gp, gdt, gst, gsh,
        block_scale, res_scale, hp, hdt, ldh, op, ldo, nxt, nw, *outs)


def matmul_i8(xq, x_scale, wq, w_scale, out, bias=None, stream=None):
    """out [T, N] = (xq [T, K] . wq [N, K]) * x_scale [T] * w_scale [N] (+ bias [N] fp32): int8 codes, exact
    int32 sums, out fp32 or bf16."""
    dev, T, K, xp, _, ldx = _first("xq", xq, "int8")
    N = wq.shape[0]
    wp, _, ldw = _mat("wq", wq, N, K, dev, "int8")
    op, odt, ldo = _mat("out", out, T, N, dev)
    _on(dev, stream, _lib.moe_matmul_i8, xp, ldx, _vec("x_scale", x_scale, T, dev, F32)[0], wp, ldw,
        _vec("w_scale", w_scale, N, dev, F32)[0], None if bias is None else _vec("bias", bias, N, dev, F32)[0], T, N, K,
        op, odt, ldo)


def gated_matmul_i8(xq, x_scale, wq, w_scale, act: int, out, stream=None):
    """out [T, F] = act(gate) * up of the int8 product of xq [T, K] with wq [2F, K] (gate rows, then up rows,
    as an expert's w13)."""
    dev, T, K, xp, _, ldx = _first("xq", xq, "int8")
    N2 = wq.shape[0]
    if N2 % 2:
        raise ValueError(f"wq has {N2} rows: gate and up rows come in pairs")
    wp, _, ldw = _mat("wq", wq, N2, K, dev, "int8")
    op, odt, ldo = _mat("out", out, T, N2 // 2, dev)
    _on(dev, stream, _lib.moe_gated_matmul_i8, xp, ldx, _vec("x_scale", x_scale, T, dev, F32)[0], wp, ldw,
        _vec("w_scale", w_scale, N2, dev, F32)[0], T, N2 // 2, K, act, op, odt, ldo)

"""Refusals of the operators around the expert FFN, without a GPU: the C ABI checks its
arguments before it enqueues anything (these calls never reach the HIP runtime), and
the binding refuses tensors it cannot pass on."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p
A = [P((i + 1) << 33) for i in range(16)]     # far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    import expert_ffn_amd as lib
    if not os.path.exists(lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return lib


def off(p, n):
    return P(p.value + n)


def call(L, name, spec, **kw):
    unknown = set(kw) - {n for n, _ in spec}
    assert not unknown, unknown
    rc = getattr(L.lib(), name)(*[kw.get(n, d) for n, d in spec])
    return rc, L.lib().moe_last_error().decode()


def refused(L, name, spec, rc, text, **kw):
    got, msg = call(L, name, spec, **kw)
    assert got == rc and msg.startswith(name + ": ") and text in msg, (kw, got, msg)


ROUTE = [("logits", A[0]), ("dt", 0), ("ld", 128), ("bias", A[1]), ("T", 4), ("E", 128), ("k", 8), ("score", 0), ("G", 8),
         ("keep", 4), ("rank", 1), ("renorm", 1), ("scale", 1.0), ("ids", A[2]), ("w", A[3]), ("s", None)]


def test_route_score_refusals(L):
    r = lambda rc, text, **kw: refused(L, "moe_route_score_topk", ROUTE, rc, text, **kw)
    for n in ("logits", "ids", "w"):
        r(1, "null", **{n: None})
    r(1, "dtype", dt=2)
    r(1, "score", score=2)
    r(1, "group rank", rank=-1)
    r(2, "T=-1", T=-1)
    r(2, "E=0", E=0)
    r(2, "E=513", E=513, G=1, keep=1)
    r(2, "n_group=7", G=7)
    r(2, "n_group=128", G=128)
    r(2, "n_group=0", G=0)
    r(2, "topk_group=9", keep=9)
    r(2, "topk_group=0", keep=0)
    r(2, "k=0", k=0)
    r(2, "k=17", k=17, keep=1)            # more than the kept group's 16 experts
    r(2, "k=33", k=33)
    r(2, "row stride 127", ld=127)
    r(2, "too large", T=(1 << 24) + 1)
    for bad in (float("inf"), float("nan")):
        r(1, "scale", scale=bad)
    r(1, "aligned", logits=off(A[0], 2))
    r(1, "aligned", bias=off(A[1], 1))
    r(1, "overlap", ids=A[0])
    r(1, "overlap", w=off(A[2], 4 * 8 * 4 - 4))
    r(1, "overlap", w=A[1])
    assert call(L, "moe_route_score_topk", ROUTE, T=0, logits=None, ids=None, w=None)[0] == 0


ROUTER = [("x", A[0]), ("dt", 1), ("T", 4), ("H", 256), ("wr", A[1]), ("E", 64), ("k", 8), ("bias", None), ("score", 1),
          ("G", 1), ("keep", 1), ("rank", 0), ("renorm", 1), ("scale", 1.0), ("logits", A[2]), ("ws", A[3]),
          ("wsb", 1 << 20), ("ids", A[4]), ("w", A[5]), ("s", None)]


def test_router_score_refusals(L):
    r = lambda rc, text, **kw: refused(L, "moe_router_score_topk", ROUTER, rc, text, **kw)
    for n in ("x", "wr", "logits", "ws", "ids", "w"):
        r(1, "null", **{n: None})
    r(2, "H=100", H=100)
    r(2, "k=65", k=65)
    r(4, "ws_bytes", wsb=16)
    r(1, "16-byte", x=off(A[0], 8))
    r(1, "overlap", ws=A[2])
    r(1, "overlap", logits=A[0])
    r(2, "too large", T=1 << 24, E=512, k=2)
    assert call(L, "moe_router_score_topk", ROUTER, T=0)[0] == 0


NORM_IN = [("h", A[0]), ("hdt", 1), ("ldh", 256), ("T", 4), ("H", 256), ("w", A[1]), ("wdt", 1), ("off", 0.0), ("eps", 1e-6),
           ("x", A[2]), ("xdt", 1), ("ldx", 256), ("xq", A[3]), ("ldq", 256), ("xs", A[4]), ("s", None)]


def test_norm_in_refusals(L):
    r = lambda rc, text, **kw: refused(L, "moe_norm_in", NORM_IN, rc, text, **kw)
    r(1, "h is NULL", h=None)
    r(1, "neither", x=None, xq=None, xs=None)
    r(1, "go together", xs=None)
    r(1, "go together", xq=None)
    r(2, "T=-1", T=-1)
    r(2, "T=2097153", T=(1 << 21) + 1)
    for H in (0, 4, 100, 32776):
        r(2, f"H={H}", H=H)
    for d in ("hdt", "wdt", "xdt"):
        r(1, "dtype", **{d: 7})
    r(2, "row stride 248 of h", ldh=248)
    r(2, "row stride 248 of x", ldx=248)
    r(2, "row stride 248 of xq", ldq=248)
    r(2, "xq", ldq=(1 << 22) + 8)
    r(1, "rows of h must be 16-byte", ldh=260)
    r(1, "rows of h must be 16-byte", h=off(A[0], 8))
    r(1, "rows of x must be 16-byte", ldx=260)
    r(1, "rows of xq must be 8-byte", ldq=260)
    r(1, "16-byte", w=off(A[1], 8))
    r(1, "4-byte", xs=off(A[4], 2))
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        r(1, "eps", eps=eps)
    r(1, "w_offset", off=float("nan"))
    r(1, "overlaps an input", x=A[0])
    r(1, "overlaps an input", xq=off(A[0], 4 * 256 * 2 - 8))
    r(1, "overlaps an input", x=A[1])
    r(1, "two outputs", xq=A[2])
    assert call(L, "moe_norm_in", NORM_IN, T=0, h=None)[0] == 0


QUANT = [("x", A[0]), ("dt", 0), ("ldx", 64), ("T", 3), ("K", 64), ("xq", A[1]), ("ldq", 64), ("xs", A[2]), ("s", None)]


def test_quantize_tokens_refusals(L):
    r = lambda rc, text, **kw: refused(L, "moe_quantize_tokens", QUANT, rc, text, **kw)
    for n in ("x", "xq", "xs"):
        r(1, "null", **{n: None})
    r(2, "K=60", K=60)
    r(1, "dtype", dt=3)
    r(2, "row stride 60 of x", ldx=60)
    r(1, "overlaps", xq=A[0])
    r(1, "overlap", xs=A[1])


NORM_OUT = [("routes", A[0]), ("rdt", 0), ("tw", A[1]), ("pos", A[2]), ("k", 2), ("y", A[3]), ("ydt", 1), ("ldy", 64), ("T", 4),
            ("H", 64), ("wp", A[4]), ("wdt", 1), ("off", 0.0), ("eps", 1e-6), ("gate", A[5]), ("gdt", 0), ("gst", 0),
            ("gsh", 1), ("bs", 1.0), ("rs", 1.0), ("h", A[6]), ("hdt", 1), ("ldh", 64), ("ho", A[7]), ("ldho", 64),
            ("next", 1), ("wn", A[8]), ("x", A[9]), ("xdt", 1), ("ldx", 64), ("xq", A[10]), ("ldq", 64), ("xs", A[11]),
            ("s", None)]


def test_norm_out_refusals(L):
    r = lambda rc, text, **kw: refused(L, "moe_norm_out", NORM_OUT, rc, text, **kw)
    r(1, "h or h_out", h=None)
    r(1, "h or h_out", ho=None)
    for n in ("routes", "tw", "pos"):
        r(1, "routes", **{n: None})
    r(1, "neither routes nor y", k=0, y=None)
    r(2, "k=33", k=33)
    r(2, "k=-1", k=-1)
    r(2, "H=60", H=60)
    for d in ("rdt", "ydt", "wdt", "gdt", "hdt", "xdt"):
        r(1, "dtype", **{d: 5})
    r(1, "eps", eps=0.0)
    r(1, "NaN", bs=float("nan"))
    r(1, "NaN", rs=float("nan"))
    r(3, "neither 0 nor 1", gsh=2)
    r(2, "gate stride", gst=-64)
    r(1, "rows of gate", gate=off(A[5], 4))
    r(1, "rows of gate", gst=66)
    r(1, "rows of h must", ldh=68)
    r(1, "rows of h_out must", ldho=68)
    r(1, "rows of y must", ldy=68)
    r(1, "out_routes", routes=off(A[0], 4))
    r(1, "w_post", wp=off(A[4], 2))
    r(1, "weight is not 16-byte", wn=off(A[8], 2))
    r(1, "outputs of the next norm", next=0)
    r(1, "neither x nor xq", x=None, xq=None, xs=None)
    r(1, "overlaps an input", ho=off(A[6], 16))          # h_out beside h, but not h itself
    r(1, "overlaps an input", ho=A[6], ldho=72)
    r(1, "overlaps an input", ho=A[3])
    r(1, "overlaps an input", x=A[0])
    r(1, "overlaps an input", xs=A[2])
    r(1, "two outputs", x=A[7])
    assert call(L, "moe_norm_out", NORM_OUT, T=0)[0] == 0


MM = [("xq", A[0]), ("ldx", 64), ("sx", A[1]), ("wq", A[2]), ("ldw", 64), ("sw", A[3]), ("bias", None), ("T", 4), ("N", 32),
      ("K", 64), ("out", A[4]), ("odt", 1), ("ldo", 32), ("s", None)]
GATED = [("xq", A[0]), ("ldx", 64), ("sx", A[1]), ("wq", A[2]), ("ldw", 64), ("sw", A[3]), ("T", 4), ("N", 32), ("K", 64),
         ("act", 0), ("out", A[4]), ("odt", 1), ("ldo", 32), ("s", None)]


@pytest.mark.parametrize("name,spec", [("moe_matmul_i8", MM), ("moe_gated_matmul_i8", GATED)])
def test_matmul_refusals(L, name, spec):
    r = lambda rc, text, **kw: refused(L, name, spec, rc, text, **kw)
    for n in ("xq", "sx", "wq", "sw", "out"):
        r(1, "null", **{n: None})
    r(2, "T=-1", T=-1)
    r(2, "N=0", N=0)
    r(2, "N=16777217", N=(1 << 24) + 1, ldo=1 << 25)
    for K in (0, 8, 72, 131072):
        r(2, f"K={K}", K=K, ldx=1 << 18, ldw=1 << 18)
    r(2, "row strides", ldx=48)
    r(2, "row strides", ldw=(1 << 22) + 16)
    r(1, "16-byte", ldx=72)
    r(1, "16-byte", wq=off(A[2], 8))
    r(2, "row stride 31 of out", ldo=31)
    r(1, "dtype", odt=4)
    r(1, "aligned", out=off(A[4], 1))
    r(1, "aligned", sx=off(A[1], 2))
    r(2, "too large", T=(1 << 24) + 1)
    r(2, "too large", T=1 << 24, N=1 << 13, ldo=1 << 13)
    r(1, "overlaps an input", out=A[0])
    r(1, "overlaps an input", out=A[3])
    assert call(L, name, spec, T=0, xq=None, out=None)[0] == 0


def test_gated_matmul_activation(L):
    refused(L, "moe_gated_matmul_i8", GATED, 1, "activation", act=2)
    # the up rows count: an output among them is an overlap
    refused(L, "moe_gated_matmul_i8", GATED, 1, "overlaps an input", out=off(A[2], 40 * 64))


def test_binding_needs_gpu_tensors(L):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt)
    i8 = torch.int8
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.route_score_topk(z(2, 8), 2, z(2, 2, dt=torch.int32), z(2, 2))
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.norm_in(z(2, 64), None, 1e-6, x=z(2, 64))
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.quantize_tokens(z(2, 64), z(2, 64, dt=i8), z(2))
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.norm_out(z(2, 64), z(2, 64), None, 1e-6, y=z(2, 64))
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.matmul_i8(z(2, 64, dt=i8), z(2), z(4, 64, dt=i8), z(4), z(2, 4))
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.gated_matmul_i8(z(2, 64, dt=i8), z(2), z(4, 64, dt=i8), z(4), 0, z(2, 2))
    with pytest.raises(ValueError, match="a GPU is needed"):
        L.router_score_topk(z(2, 64), z(8, 64), 2, z(2, 8), z(64), z(2, 2, dt=torch.int32), z(2, 2))


def test_dense_expert_blob_size(L):
    from expert_ffn_amd.layer import DenseExpert
    n = L.expert_bytes(L.W_INT8_ROW, 128, 64)
    d = DenseExpert(torch.zeros(n, dtype=torch.uint8), 128, 64)
    o = L.blob_layout(L.W_INT8_ROW, 128, 64)
    base = d.blob.data_ptr()
    assert [d.w13.data_ptr() - base, d.s13.data_ptr() - base, d.w2.data_ptr() - base, d.s2.data_ptr() - base] == o[:4]
    assert d.w13.shape == (128, 128) and d.w2.shape == (128, 64) and d.s13.shape == (128,) and d.s2.shape == (128,)
    with pytest.raises(ValueError, match="blob"):
        DenseExpert(torch.zeros(n - 1, dtype=torch.uint8), 128, 64)


def test_bound_functions():
    """The compiled binding: names and signatures as documented, and its own argument errors (no GPU needed)."""
    import inspect

    import expert_ffn_amd as lib
    want = {"route_score_topk": 12, "router_score_topk": 15, "norm_in": 8, "quantize_tokens": 4, "norm_out": 17, "matmul_i8": 7,
            "gated_matmul_i8": 7}
    for name, n in want.items():
        assert len(inspect.signature(getattr(lib, name)).parameters) == n
    with pytest.raises(AttributeError):
        lib.no_such_function
    h = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="a GPU is needed"):
        lib.norm_in(h, None, 1e-6, x=h)
    with pytest.raises(TypeError, match="missing its argument 'eps'"):
        lib.norm_in(h, None)
    with pytest.raises(TypeError, match="unexpected keyword argument 'y'"):
        lib.norm_in(h, None, 1e-6, y=h)
    with pytest.raises(TypeError, match="multiple values for argument 'w'"):
        lib.norm_in(h, None, 1e-6, w=None)
    with pytest.raises(TypeError, match="takes 4 arguments"):
        lib.quantize_tokens(h, h, h, None, None)
    with pytest.raises(TypeError, match="h is not a tensor"):
        lib.norm_in(None, None, 1e-6)


def test_layer_imports_without_the_library(tmp_path):
    """Nothing of the package is loaded before the first call; then a missing build raises."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import expert_ffn_amd as lib\n"
            f"lib.LIB_PATH = {str(tmp_path / 'none.so')!r}\n"
            "import expert_ffn_amd.layer\n"
            "try:\n    lib.norm_in\nexcept ImportError as e:\n    print('refused:', e)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120, cwd=root)
    assert r.returncode == 0 and "refused:" in r.stdout and "is missing" in r.stdout, r.stdout + r.stderr

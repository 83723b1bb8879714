"""Refusals of the bfloat16 products, their backward passes and the adapters, without a GPU: the C
ABI checks its arguments before it enqueues anything, and the binding refuses tensors it cannot pass on."""
import pytest
import torch

from test_block_abi import A, call, off, refused
from test_block_abi import L  # noqa: F401  (the fixture)

AD = [("sh", None), ("lds", 0), ("ids", None), ("b", None), ("bs", 0), ("ranks", None), ("n", 0), ("R", 0), ("s", None)]
MM = [("x", A[0]), ("ldx", 64), ("w", A[1]), ("ldw", 64), ("T", 5), ("N", 100), ("K", 64), ("out", A[2]), ("odt", 1), ("ldo", 100)] + AD
GM = [("x", A[0]), ("ldx", 64), ("w", A[1]), ("ldw", 64), ("T", 5), ("N", 100), ("K", 64), ("act", 0), ("out", A[2]), ("odt", 1),
      ("ldo", 100), ("pre", A[3]), ("ldp", 200)] + AD
SHRINK = [("x", A[0]), ("ldx", 64), ("T", 5), ("K", 64), ("ids", A[1]), ("a", A[2]), ("as", 2 * 16 * 64), ("n", 3), ("R", 16),
          ("halves", 2), ("scale", A[3]), ("ranks", A[4]), ("sh", A[5]), ("lds", 32), ("s", None)]
MMB = [("x", A[0]), ("ldx", 64), ("w", A[1]), ("ldw", 64), ("d", A[2]), ("ldd", 104), ("T", 5), ("N", 104), ("K", 64), ("dx", A[3]),
       ("xdt", 1), ("lddx", 64), ("dw", A[4]), ("wdt", 0), ("lddw", 64), ("s", None)]
GMB = [("x", A[0]), ("ldx", 64), ("w", A[1]), ("ldw", 64), ("act", 1), ("pre", A[5]), ("ldp", 208), ("d", A[2]), ("ldd", 104), ("T", 5),
       ("N", 104), ("K", 64), ("dp", A[6]), ("ldg", 208), ("dx", A[3]), ("xdt", 1), ("lddx", 64), ("dw", A[4]), ("wdt", 0), ("lddw", 64),
       ("s", None)]
BIG = 1 << 21


def with_adapters(rows):
    R = 16
    return dict(sh=A[8], lds=2 * R, ids=A[9], b=A[10], bs=rows * R, ranks=A[11], n=3, R=R)


@pytest.mark.parametrize("name,spec,rows", [("moe_matmul_bf16", MM, 100), ("moe_gated_matmul_bf16", GM, 200)])
def test_product_refusals(L, name, spec, rows):  # noqa: F811
    r = lambda rc, text, **kw: refused(L, name, spec, rc, text, **kw)
    for n in ("x", "w", "out"):
        r(1, "null", **{n: None})
    r(2, "T=-1", T=-1)
    r(2, "T=", T=(1 << 24) + 1)
    r(2, "=0 outside", N=0)
    for K in (0, 4, 60, (1 << 20) + 8):
        r(2, "K=", K=K, ldx=BIG, ldw=BIG)
    r(2, "too large", T=1 << 20, N=1 << 17, ldo=1 << 18, **({"ldp": 1 << 18} if spec is GM else {}))
    r(2, "row stride", ldx=56)
    r(2, "row stride", ldw=BIG + 8)
    r(2, "row stride", ldo=99)
    r(2, "too large", ldo=1 << 40)
    r(1, "aligned", ldx=68)
    r(1, "aligned", x=off(A[0], 8))
    r(1, "aligned", w=off(A[1], 2))
    r(1, "aligned", out=off(A[2], 1))
    r(1, "aligned", out=off(A[2], 2), odt=0)
    r(1, "dtype", odt=2)
    r(1, "overlap", out=off(A[0], 16))
    r(1, "overlap", out=off(A[1], 64 * 2 * (rows - 1)))
    ad = with_adapters(rows)
    r(1, "go with s", ids=A[9])
    r(1, "go with s", b=A[10])
    r(1, "null", **dict(ad, ids=None))
    r(1, "null", **dict(ad, b=None))
    r(2, "n_adapters=0", **dict(ad, n=0))
    for R in (0, 4, 20, 1032):
        r(2, "R=", **dict(ad, R=R, bs=rows * 2048, lds=4096))
    r(2, "stride", **dict(ad, bs=rows * 16 - 8))
    r(2, "stride", **dict(ad, bs=1 << 40))
    r(1, "aligned", **dict(ad, bs=rows * 16 + 4))
    r(1, "aligned", **dict(ad, b=off(A[10], 8)))
    r(1, "aligned", **dict(ad, sh=off(A[8], 4)))
    r(1, "aligned", **dict(ad, ids=off(A[9], 2)))
    r(2, "row stride", **dict(ad, lds=8))
    r(1, "overlap", **dict(ad, sh=A[2]))
    r(1, "overlap", **dict(ad, ids=A[2]))
    r(1, "overlap", **dict(ad, out=off(A[10], 2 * 2 * rows * 16)))
    assert call(L, name, spec, T=0, x=None, out=None)[0] == 0
    if spec is GM:
        r(1, "activation", act=2)
        r(1, "overlap", pre=A[2])
        r(1, "aligned", pre=off(A[3], 1))
        r(2, "row stride", ldp=199)


def test_shrink_refusals(L):  # noqa: F811
    r = lambda rc, text, **kw: refused(L, "moe_adapter_shrink", SHRINK, rc, text, **kw)
    for n in ("x", "ids", "a", "sh"):
        r(1, "null", **{n: None})
    r(2, "T=-1", T=-1)
    r(2, "K=", K=60)
    r(1, "halves=3", halves=3)
    r(1, "halves=0", halves=0)
    r(2, "n_adapters=0", n=0)
    for R in (12, 1032):
        r(2, "R=", R=R, **{"as": 1 << 20, "lds": 4096})
    r(2, "stride", **{"as": 2 * 16 * 64 - 8})
    r(1, "aligned", **{"as": 2 * 16 * 64 + 4})
    r(2, "row stride", lds=24)
    r(1, "aligned", lds=36)
    r(1, "aligned", scale=off(A[3], 2))
    r(1, "overlap", sh=A[0])
    r(1, "overlap", sh=A[3])
    assert call(L, "moe_adapter_shrink", SHRINK, T=0, x=None, sh=None)[0] == 0


@pytest.mark.parametrize("name,spec", [("moe_matmul_bf16_backward", MMB), ("moe_gated_matmul_bf16_backward", GMB)])
def test_backward_refusals(L, name, spec):  # noqa: F811
    r = lambda rc, text, **kw: refused(L, name, spec, rc, text, **kw)
    for n in ("x", "w", "d"):
        r(1, "null", **{n: None})
    r(2, "T=-1", T=-1)
    r(2, "K=", K=60)
    r(2, "not a multiple of 8", N=100)
    for n in ("ldx", "ldw", "ldd", "lddx", "lddw"):
        r(2, "row stride", **{n: 56})
    for n in ("ldx", "ldw", "ldd"):
        r(1, "aligned", **{n: 108})
    r(1, "dtype", xdt=2)
    r(1, "dtype", wdt=-1)
    r(1, "aligned", dx=off(A[3], 1))
    r(1, "aligned", dw=off(A[4], 2))
    r(1, "overlap", dw=A[3])
    r(1, "overlap", dx=A[2])
    r(1, "overlap", dw=A[0])
    if spec is MMB:
        r(1, "neither", dx=None, dw=None)
        return
    r(1, "activation", act=-1)
    for n in ("pre", "dp"):
        r(1, "null", **{n: None})
    r(2, "row stride", ldp=200)
    r(1, "aligned", dp=off(A[6], 2))
    r(1, "overlap", dp=A[2])
    r(1, "overlap", dp=off(A[5], 16))        # pre itself, or apart from it
    r(1, "overlap", dx=A[6])


@pytest.mark.parametrize("name,spec,half", [("moe_matmul_bf16_backward", MMB, 1), ("moe_gated_matmul_bf16_backward", GMB, 2)])
def test_backward_refuses_gradients_that_no_launch_takes(L, name, spec, half):  # noqa: F811
    """Before the activation's gradient is enqueued: dx or dw of more than 2^36 elements."""
    r = lambda text, **kw: refused(L, name, spec, 2, text, **kw)
    K = 1 << 17
    wide = dict(K=K, ldx=K, ldw=K, lddx=K, lddw=K)
    r("of dx too large", T=(1 << 19) + 1, **wide)
    r("of dw too large", N=(1 << 19) // half + 8, ldd=1 << 20, dx=None, **wide, **(dict(ldp=1 << 21, ldg=1 << 21) if half == 2 else {}))


def test_binding_refusals(L):  # noqa: F811
    """Tensors on the host, and arguments that do not go together."""
    x, w, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 64), (32, 64), (4, 32)))
    for f, a in ((L.matmul_bf16, (x, w, y)), (L.gated_matmul_bf16, (x, w, 0, y)), (L.matmul_bf16_backward, (x, w, y)),
                 (L.gated_matmul_bf16_backward, (x, w, 0, y, y, y)), (L.adapter_shrink, (x, None, w, None, y))):
        with pytest.raises(ValueError, match="x is on cpu"):
            f(*a)
        with pytest.raises(TypeError, match="unexpected keyword"):
            f(*a, nothing=1)
        with pytest.raises(TypeError, match="missing"):
            f(x)


def test_experts_and_adapters_refuse_what_does_not_fit(L):  # noqa: F811
    from expert_ffn_amd.layer import Adapters, DenseExpertBf16
    H, FF = 128, 64
    n = L.expert_bytes(L.W_BF16, H, FF)
    blob = torch.zeros(n, dtype=torch.uint8)
    e = DenseExpertBf16(blob, H, FF, adapters=Adapters(3, 16, H, FF, "cpu"))
    assert e.w13.shape == (2 * FF, H) and e.w2.shape == (H, FF)
    for bad in (blob[:n - 1], blob.view(torch.int8), torch.zeros(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous bytes"):
            DenseExpertBf16(bad, H, FF)
    with pytest.raises(ValueError, match="the adapters have"):
        DenseExpertBf16(blob, H, FF, adapters=Adapters(3, 16, H, FF + 8, "cpu"))
    for n_, R in ((0, 16), (3, 0), (3, 12), (3, 1032)):
        with pytest.raises(ValueError, match="R="):
            Adapters(n_, R, H, FF, "cpu")
    parts = lambda r, F=FF: [torch.ones(s) for s in ((2, r, H), (2 * F, r), (r, F), (H, r))]
    with pytest.raises(ValueError, match="slot 3"):
        e.adapters.load(3, *parts(16))
    for p in (parts(17), parts(8, FF + 8), [parts(8)[0], *parts(4)[1:]]):
        with pytest.raises(ValueError, match="do not fit"):
            e.adapters.load(0, *p)
    assert not e.adapters.ranks.any()
    e.adapters.load(1, *parts(5), scale=0.5)
    assert e.adapters.ranks.tolist() == [0, 5, 0] and e.adapters.scale.tolist() == [1.0, 0.5, 1.0]
    assert e.adapters.a2[1, :5].all() and not e.adapters.a2[1, 5:].any()


def test_block_takes_other_experts_as_before(L):  # noqa: F811
    """A dense expert of the user's own, with DenseExpert's members, is one in 8 bits."""
    from expert_ffn_amd.layer import DenseExpert, DenseExpertBf16, MoeBlock, MoeLayer

    class Own:
        H, FF = 128, 64

    blob = lambda fmt: torch.zeros(L.expert_bytes(fmt, 128, 64), dtype=torch.uint8)
    make = lambda d: MoeBlock(MoeLayer(8, 2, 128, 64, L.W_BF16, 4, device="cpu"), torch.zeros(128), torch.zeros(8, 128), dense=d)
    for dense, codes in ((Own(), True), (DenseExpert(blob(L.W_INT8_ROW), 128, 64), True), (DenseExpertBf16(blob(L.W_BF16), 128, 64), False),
                         (None, False)):
        b = make(dense)
        assert b.codes == codes and hasattr(b, "xq") == codes and b.low is None

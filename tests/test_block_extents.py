"""Matrices whose last row would lie beyond any address are refused before their overlap is
checked (the check's byte counts stay inside 64 bits): the C ABI without a GPU."""
import pytest

from test_block_abi import GATED, MM, NORM_IN, NORM_OUT, QUANT, ROUTE, ROUTER, A, call, refused
from test_block_abi import L  # noqa: F401  (the fixture)

FAR = (1 << 40) - 16                       # elements from row to row
ROWS, MANY = 1 << 21, 1 << 24              # the most rows of a norm, and of a routing or a product


@pytest.mark.parametrize("name,spec,kw", [
    ("moe_route_score_topk", ROUTE, dict(T=MANY, E=1, k=1, G=1, keep=1, ld=FAR)),
    ("moe_norm_in", NORM_IN, dict(T=ROWS, ldh=FAR)),
    ("moe_norm_in", NORM_IN, dict(T=ROWS, ldx=FAR)),
    ("moe_quantize_tokens", QUANT, dict(T=ROWS, ldx=FAR)),
    ("moe_norm_out", NORM_OUT, dict(T=ROWS, ldh=FAR)),
    ("moe_norm_out", NORM_OUT, dict(T=ROWS, ldho=FAR)),
    ("moe_norm_out", NORM_OUT, dict(T=ROWS, ldy=FAR)),
    ("moe_norm_out", NORM_OUT, dict(T=ROWS, gst=FAR)),
    ("moe_norm_out", NORM_OUT, dict(T=ROWS, ldx=FAR)),
    ("moe_matmul_i8", MM, dict(T=MANY, ldo=FAR)),
    ("moe_gated_matmul_i8", GATED, dict(T=MANY, ldo=FAR)),
])
def test_rows_beyond_any_address(L, name, spec, kw):  # noqa: F811
    refused(L, name, spec, 2, "too large", **kw)
    # the same stride with few rows is an ordinary call (here one that is refused for a later reason)
    few = dict(kw, T=2)
    assert "too large" not in call(L, name, spec, **few, **{spec[0][0]: None})[1]


def test_overlap_behind_a_wrapped_extent(L):  # noqa: F811
    """2^21 rows 2^40 elements apart are 2^63 bytes: an output inside them was not seen to overlap."""
    rc, msg = call(L, "moe_norm_in", NORM_IN, T=ROWS, ldh=FAR, hdt=0, x=A[0], xq=None, xs=None)
    assert rc == 2 and "too large" in msg, (rc, msg)


def test_router_tokens_beyond_a_launch(L):  # noqa: F811
    """The router's product has a grid row per 64 tokens, at most 65535: more tokens are refused, not left to the launch."""
    few = dict(H=64, E=1, k=1, wsb=1 << 34)
    refused(L, "moe_router_score_topk", ROUTER, 2, "too large", T=65535 * 64 + 1, **few)
    assert "too large" not in call(L, "moe_router_score_topk", ROUTER, T=65535 * 64, **dict(few, wsb=16))[1]

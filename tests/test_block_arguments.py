"""Argument combinations that the compiled binding refuses before it looks at a tensor (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import os

    import expert_ffn_amd as lib
    if not os.path.exists(lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return lib


@pytest.mark.parametrize("names", [("topk_w",), ("route_pos",), ("topk_w", "route_pos")])
def test_norm_out_routes_without_their_rows(L, names):
    """Weights or positions of routes without the routes' rows: the routed experts' share would be missing."""
    h, y = torch.zeros(2, 64), torch.zeros(2, 64)
    given = {"topk_w": torch.zeros(2, 2), "route_pos": torch.zeros(2, 2, dtype=torch.int32)}
    with pytest.raises(ValueError, match="need out_routes"):
        L.norm_out(h, torch.empty_like(h), None, 1e-6, y=y, **{n: given[n] for n in names})


def test_router_workspace_grows_with_the_tokens(L):
    """The workspace of a block's largest batch is enough for its smaller ones."""
    for H in (64, 128, 192, 256, 320, 2816, 7168):
        for E in (1, 60, 128, 512):
            sizes = [L.router_ws_bytes(T, H, E) for T in (1, 2, 16, 63, 64, 65, 66, 127, 128, 1000, 16384)]
            assert sizes == sorted(sizes), (H, E, sizes)

"""The dense expert in bf16 and its adapters without a GPU: what run() and load() refuse or leave alone."""
import pytest
import torch

from test_block_abi import L  # noqa: F401  (the fixture)

H, FF, T = 128, 64, 4


def expert(L, adapters=None):  # noqa: F811
    from expert_ffn_amd.layer import DenseExpertBf16
    return DenseExpertBf16(torch.zeros(L.expert_bytes(L.W_BF16, H, FF), dtype=torch.uint8), H, FF, adapters=adapters)


def test_sums_for_the_backward_pass_are_refused_with_adapters(L):  # noqa: F811
    """backward() has no adapter terms: run() does not store the sums of a pass with adapters for it."""
    from expert_ffn_amd.layer import Adapters
    new = lambda c, dt=torch.bfloat16: torch.zeros(T, c, dtype=dt)
    x, hid, y, pre, low, ids = new(H), new(FF), new(H), new(2 * FF), new(32), torch.zeros(T, dtype=torch.int32)
    e = expert(L, Adapters(3, 16, H, FF, "cpu"))
    with pytest.raises(ValueError, match="pre goes with a pass without adapters"):
        e.run(x, hid, y, pre=pre, low=low, adapter_ids=ids)
    # either alone passes these checks (and ends at the tensors, which are on the host)
    for more in (dict(pre=pre), dict(low=low, adapter_ids=ids), dict(pre=pre, low=low)):
        with pytest.raises(ValueError, match="x is on cpu"):
            e.run(x, hid, y, **more)


def test_loaded_adapters_leave_no_graph(L):  # noqa: F811
    """Adapters are often parameters of a training program: the pools stay plain buffers."""
    from expert_ffn_amd.layer import Adapters
    a = Adapters(2, 16, H, FF, "cpu")
    parts = [torch.nn.Parameter(torch.full(s, 0.5)) for s in ((2, 8, H), (2 * FF, 8), (8, FF), (H, 8))]
    scale = torch.tensor(2.0, requires_grad=True)
    for slot in (1, 0, 1):
        a.load(slot, *parts, scale=scale * 3)
    for t in (a.a13, a.b13, a.a2, a.b2, a.scale, a.ranks):
        assert not t.requires_grad and t.grad_fn is None
    assert a.ranks.tolist() == [8, 8] and a.scale.tolist() == [6.0, 6.0]
    assert (a.b13[1, :, :8] == 0.5).all() and not a.b13[1, :, 8:].any()


def block(L, dense):  # noqa: F811
    from expert_ffn_amd.layer import MoeBlock, MoeLayer
    return MoeBlock(MoeLayer(8, 2, H, 64, L.W_BF16, T, device="cpu"), torch.zeros(H), torch.zeros(8, H), dense=dense)


def test_block_asks_only_the_bf16_expert_for_adapters(L):  # noqa: F811
    """A dense expert of the user's own may have any member of that name."""
    from expert_ffn_amd.layer import Adapters

    class Own:
        H, FF, adapters = 128, 64, ["of", "its", "own"]

    b = block(L, Own())
    assert b.codes and b.low is None
    with pytest.raises(ValueError, match="no adapters"):
        b.run(torch.zeros(T, H), torch.zeros(T, H), adapter_ids=torch.zeros(T, dtype=torch.int32))
    assert block(L, expert(L, Adapters(3, 16, H, FF, "cpu"))).low.shape == (T, 32)
    assert block(L, expert(L)).low is None


def test_run_dense_refuses_ids_that_no_adapter_takes(L):  # noqa: F811
    """Called by itself, with an expert in 8 bits: the ids were left out without a word."""
    from expert_ffn_amd.layer import DenseExpert
    d = DenseExpert(torch.zeros(L.expert_bytes(L.W_INT8_ROW, H, FF), dtype=torch.uint8), H, FF)
    ids = torch.zeros(T, dtype=torch.int32)
    for dense in (d, expert(L), None):
        with pytest.raises(ValueError, match="no adapters"):
            block(L, dense).run_dense(T, adapter_ids=ids)

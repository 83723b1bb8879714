"""The norms around the block on the GPU at arguments between the ordinary ones: gates of one value per
row in both types, at any stride and alignment of their elements."""
import numpy as np
import pytest
import torch

import block_ref as ref
from block_ref import f64, half_step
from test_gpu_block import BF16, EPS, F32, L, close, gen, normal  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gt", [BF16, F32])
@pytest.mark.parametrize("T,H", [(1, 64), (5, 520), (33, 2816), (3, 16392)])
@pytest.mark.parametrize("layout", ["column", "strided", "odd start", "one", "scalar"])
def test_gate_of_one_value_per_row(L, T, H, gt, layout):  # noqa: F811
    g = gen(T + H)
    values = normal(g, T + 2, 3, dtype=gt)
    gate = {"column": values[:T, :1].contiguous(), "strided": values[:T, 1:2], "odd start": values.view(-1)[1:1 + T].view(T, 1),
            "one": values[:1, 2:3], "scalar": values[1, 1]}[layout]
    h, y = normal(g, T, H, dtype=BF16), normal(g, T, H)
    wp, wn = normal(g, H, dtype=BF16), normal(g, H, dtype=BF16)
    ho, x, x2 = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    L.norm_out(h, ho, wp, EPS, y=y, gate=gate, block_scale=0.5, w_next=wn, x=x)
    want, bound = ref.norm_out(f64(h), None, None, None, f64(y), f64(wp), 0.0, EPS,
                               f64(gate if gate.dim() else gate.view(1, 1)), 0.5, 1.0)
    close(f64(ho), want, bound + half_step(BF16) * (np.abs(want) + bound), "h_out")
    # the same gate as a full matrix: the same bits
    full = gate.expand(T, H).contiguous()
    ho2 = torch.empty_like(h)
    L.norm_out(h, ho2, wp, EPS, y=y, gate=full, block_scale=0.5, w_next=wn, x=x2)
    assert torch.equal(ho, ho2) and torch.equal(x, x2)

"""Ranks outside [0, R] count as the nearest of the two, to the ends of their type: what an adapter's B holds
past its rank is not used (few tokens and tiles)."""
import pytest
import torch

from bf16_ref import BF16, F32, F64, adapters, whole
from test_gpu_bf16 import equal
from test_gpu_block import L, check_padding, gen, padded  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu
LOW, HIGH = -(1 << 31), (1 << 31) - 1


# up to 64 tokens the kernels for few tokens take these sizes (at most 656 weight rows), then tiles
@pytest.mark.parametrize("T", [1, 16, 17, 40, 61, 129, 700])
@pytest.mark.parametrize("R", [8, 32, 72])
@pytest.mark.parametrize("gated", [False, True])
def test_ranks_to_the_ends_of_their_type(L, T, R, gated):  # noqa: F811
    N, K, halves = 328, 264, 2 if gated else 1
    print(f"[case] ranks T={T} R={R} gated={gated}", flush=True)
    g = gen(T + R)
    r = [LOW, LOW + 1, LOW + 8, LOW + 15, LOW + 23, LOW + R, -1, 0, 3, R, R + 1, HIGH - R, HIGH]
    ranks = torch.tensor(r, dtype=torch.int32, device="cuda")
    n = len(r)
    x, w = whole(g, T, K, top=1), whole(g, halves * N, K)
    a, b = whole(g, n, halves, R, K, top=1), whole(g, n, halves * N, R)
    x = (x.float() * (torch.rand((T, K), generator=g, device="cuda") < 0.5)).to(BF16)
    past = torch.arange(R, device="cuda")[None, :] >= ranks[:, None]
    low_a, low_b = a, b
    a = torch.where(past[:, None, :, None], torch.full_like(a, float("nan")), a)
    b = torch.where(past[:, None, :], torch.full_like(b, float("inf")), b)
    for first in range(0, n, T) if T < n else (0,):   # every rank meets a token
        ids = ((torch.arange(T, device="cuda") + first) % n).to(torch.int32)
        low, up = adapters(x, ids, low_a, low_b, None, ranks, halves)
        assert low.abs().max() <= 256
        s, sbuf = padded(T, halves * R, BF16, 8, 2.0)
        L.adapter_shrink(x, ids, a if gated else a[:, 0], None, s, ranks=ranks)
        torch.cuda.synchronize()
        check_padding(sbuf, halves * R, 2.0)
        equal(s, low, "s")
        v = x.to(F64) @ w.to(F64).t().contiguous() + up
        out, buf = padded(T, N, F32, 3, 2.0)
        if gated:
            pre, pbuf = padded(T, 2 * N, BF16, 1, 2.0)
            L.gated_matmul_bf16(x, w, 1, out, pre=pre, s=s, adapter_ids=ids, b=b, ranks=ranks)
            torch.cuda.synchronize()
            check_padding(pbuf, 2 * N, 2.0)
            equal(pre, v, "pre")
        else:
            L.matmul_bf16(x, w, out, s=s, adapter_ids=ids, b=b, ranks=ranks)
            torch.cuda.synchronize()
            equal(out, v, "out")
        check_padding(buf, N, 2.0)

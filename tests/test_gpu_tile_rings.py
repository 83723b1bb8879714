"""The 8-bit products on the GPU at shapes whose rings of stages run around (tile_cases.py): the copies into
buffers that were just read, and the waits for them, in every kernel."""
import pytest
import torch

import block_ref as ref
import tile_cases as tc
from block_ref import f64, half_step
from test_gpu_block import BF16, F32, L, check_padding, close, gen, padded, rand_codes  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu


def output(T, N, bf16, pieces):
    """A padded output whose rows are 16-byte aligned, or are not."""
    pad = 8 + -N % 8 if pieces else 3 + N % 2      # a stride of whole pieces, or an odd one
    out, buf = padded(T, N, BF16 if bf16 else F32, pad, 2.0)
    assert (out.data_ptr() % 16 == 0 and out.stride(0) * out.element_size() % 16 == 0) == pieces
    return out, buf


@pytest.mark.parametrize("T,N,K,bf16,pieces", tc.PLAIN)
def test_matmul_ring(L, T, N, K, bf16, pieces):  # noqa: F811
    print(f"[case] matmul_i8 T={T} N={N} K={K} {tc.kernel_of(T, N, K, False)}", flush=True)
    g = gen(T + N + K)
    xq, wq = rand_codes(g, T, K, 16), rand_codes(g, N, K, 32)
    sx, sw = (torch.rand(n, generator=g, device="cuda") * 0.01 for n in (T, N))
    out, buf = output(T, N, bf16, pieces)
    L.matmul_i8(xq, sx, wq, sw, out)
    torch.cuda.synchronize()
    check_padding(buf, N, 2.0)
    want, bound = ref.matmul_i8(xq.cpu().numpy(), f64(sx), wq.cpu().numpy(), f64(sw))
    close(f64(out), want, bound + half_step(out.dtype) * (abs(want) + bound), "out")


@pytest.mark.parametrize("T", [49, 64])
@pytest.mark.parametrize("past", [0, 16])
def test_switch_of_64_tokens_by_length(L, T, past):  # noqa: F811
    """49 to 64 tokens at the longest rows of the kernel for few tokens, and one piece past them."""
    K = tc.FEW_STEPS_64 * tc.STEP + past
    assert (tc.kernel_of(T, 1003, K, False)[0] == ("few", 4)) == (past == 0)
    test_matmul_ring(L, T, 1003, K, True, False)
    test_gated_matmul_ring(L, T, 1003, K, False, True)


@pytest.mark.parametrize("T,F,K,bf16,pieces", tc.GATED)
def test_gated_matmul_ring(L, T, F, K, bf16, pieces):  # noqa: F811
    print(f"[case] gated_matmul_i8 T={T} F={F} K={K} {tc.kernel_of(T, F, K, True)}", flush=True)
    g = gen(T + F + K)
    xq, wq = rand_codes(g, T, K, 16), rand_codes(g, 2 * F, K, 16)
    s = 3.0 / (73.0 * 73.0 * K ** 0.5)      # products of order 1 to 3
    sx = (0.2 + torch.rand(T, generator=g, device="cuda")) * s
    sw = 0.2 + torch.rand(2 * F, generator=g, device="cuda")
    out, buf = output(T, F, bf16, pieces)
    act = F % 2
    L.gated_matmul_i8(xq, sx, wq, sw, act, out)
    torch.cuda.synchronize()
    check_padding(buf, F, 2.0)
    v, _ = ref.matmul_i8(xq.cpu().numpy(), f64(sx), wq.cpu().numpy(), f64(sw))
    want, bound = ref.gated(v[:, :F], v[:, F:], act)
    close(f64(out), want, bound + half_step(out.dtype) * (abs(want) + bound), "out")

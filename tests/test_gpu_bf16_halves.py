"""Gate's sums take gate's half of s only, up's the other: what one half holds, an infinity or NaN included,
does not reach the sums of the other (few tokens and tiles)."""
import pytest
import torch

from bf16_ref import BF16, F32, F64, whole
from test_gpu_block import L, check_padding, gen, padded  # noqa: F401  (L is the fixture)

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


# up to 64 tokens the kernels for few tokens take these sizes (656 weight rows), then tiles with and without K groups
@pytest.mark.parametrize("T", [1, 16, 17, 40, 61, 129, 700])
@pytest.mark.parametrize("R", [8, 40])
@pytest.mark.parametrize("broken", [0, 1])
def test_halves_do_not_meet(L, T, R, broken):  # noqa: F811
    n, F, K = 5, 328, 264
    print(f"[case] halves T={T} R={R} broken={broken}", flush=True)
    g = gen(T + R)
    x, w, b = whole(g, T, K, top=1), whole(g, 2 * F, K), whole(g, n, 2 * F, R)
    ids = (torch.arange(T, device="cuda") % n).to(torch.int32)
    s = whole(g, T, 2 * R, top=3)
    at = broken * R
    s[0::3, at + R - 1] = INF
    s[1::3, at] = -INF
    s[2::5, at + 3] = NAN
    out, buf = padded(T, F, F32, 3, 2.0)
    pre, pbuf = padded(T, 2 * F, BF16, 1, 2.0)
    L.gated_matmul_bf16(x, w, 1, out, pre=pre, s=s, adapter_ids=ids, b=b)
    torch.cuda.synchronize()
    check_padding(buf, F, 2.0)
    check_padding(pbuf, 2 * F, 2.0)
    v = x.cpu().to(F64) @ w.cpu().to(F64).t().contiguous()
    for h in range(2):
        sh, cols = s[:, h * R:(h + 1) * R].cpu().to(F64), slice(h * F, (h + 1) * F)
        for k in range(n):
            v[k::n, cols] += sh[k::n] @ b[k, cols].cpu().to(F64).t().contiguous()
    # sums of whole numbers are exact; infinities and NaN as the definition's (an infinity times 0 is NaN)
    want = v.to(F32).to(BF16).cuda()
    whole_half, other = (slice(F, 2 * F), slice(0, F)) if broken == 0 else (slice(0, F), slice(F, 2 * F))
    assert torch.isfinite(want[:, whole_half]).all() and not torch.isfinite(want[0, other]).all()
    for what, cols in (("the whole half", whole_half), ("the broken half", other)):
        same = (pre[:, cols] == want[:, cols]) | (pre[:, cols].isnan() & want[:, cols].isnan())
        assert same.all(), (what, int((~same).sum()), (~same).nonzero()[:5].tolist())
    # an infinite up, or a gate of +infinity (its activation is the gate), gives an infinite product
    gate, up = want[:, :F].float(), want[:, F:].float()
    far = (torch.isinf(up) & (gate > 0)) | ((gate == INF) & (up != 0) & ~up.isnan())
    assert far.any() and torch.equal(out[far], (gate * up)[far])

"""Sums of the gated projections that leave FP32's range: what is kept of them is infinite or NaN, whole blocks of
codes at a time, and no other row or block changes."""
import pytest
import torch

import gated_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def n(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


# every kernel of the projections: up to 8 rows, parts that are joined, each tile size
SHAPES = [(3, 72, 264), (40, 72, 4104), (300, 72, 264), (3000, 1032, 64), (4096, 2056, 264), (3100, 1288, 776)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_what_is_kept(gpu, M, N, K, sign):
    x, w, row, over = n(M, K), n(2 * N, K, seed=1, scale=K ** -0.5).abs(), M // 2, 40
    w[over:N], w[N + over:] = 0.0, 0.0                 # the other outputs are zero
    b = n(2 * N, seed=2)
    calm = gpu.glu_gated_linear(x, w, b, save="bf16"), gpu.glu_gated_linear(x, w, b, save="mxfp8")
    x[row] = sign * 3e38
    exact = x[row].double() @ w.double().t()
    assert (sign * exact.view(2, N)[:, :over] > 1e39).all() and (exact.view(2, N)[:, over:] == 0).all()
    others = torch.arange(M, device="cuda") != row

    h, pre, extra = gpu.glu_gated_linear(x, w, b, save="bf16")
    for kept in ref.widened(pre, extra, N):
        assert (kept[row, :over] == sign * float("inf")).all() and torch.isfinite(kept[row, over:]).all()
    assert torch.isfinite(h[row, over:].float()).all()
    if sign > 0:
        assert (h[row, :over] == float("inf")).all()
    for a, c in zip((h, pre, extra), calm[0]):
        assert torch.equal(a[others], c[others])

    h8, codes, scales = gpu.glu_gated_linear(x, w, b, save="mxfp8")
    assert torch.equal(h8.view(torch.int16), h.view(torch.int16))
    NB = (N + 31) // 32
    assert (scales[row].view(2, NB)[:, :2] == 255).all() and (scales[row].view(2, NB)[:, 2:] < 255).all()
    for kept in ref.restored(codes, scales, N):
        assert torch.isnan(kept[row, :64]).all() and torch.isfinite(kept[row, 64:]).all()
    for a, c in zip((h8, codes, scales), calm[1]):
        assert torch.equal(a[others], c[others])

    dh = n(M, N, seed=3)
    for p, e, c in ((pre, extra, calm[0]), (codes, scales, calm[1])):
        dx = gpu.glu_gated_linear_bwd(dh, x, w, p, e, need_dw=False)[0]
        assert torch.isnan(dx[row]).all()
        assert torch.equal(dx[others], gpu.glu_gated_linear_bwd(dh, x, w, *c[1:], need_dw=False)[0][others])

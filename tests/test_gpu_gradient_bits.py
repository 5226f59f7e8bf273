"""A gradient has the same bits whether the other one is formed with it or not, and with or without the bias's."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# sums that are cut into parts when formed alone, or together, or never; tiles of either size; whole and partial steps
SHAPES = [(8, 8, 8), (64, 1024, 512), (64, 2048, 128), (256, 512, 512), (300, 4096, 512), (512, 2048, 512), (512, 1504, 512),
          (1000, 1000, 1000), (1021, 2000, 2056), (2048, 1024, 512), (2048, 1024, 1024), (2000, 512, 512), (3000, 1000, 1000),
          (4096, 512, 512), (4096, 4096, 256), (4096, 4096, 512), (2048, 2048, 2048), (704, 704, 2800), (8192, 512, 264)]


def n(*shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(gpu, M, N, K):
    dy, x, w = n(M, N, seed=1), n(M, K, seed=2), n(N, K, seed=3)
    dx, dw, _ = gpu.glu_linear_bwd(dy, x, w)
    dxb, dwb, db = gpu.glu_linear_bwd(dy, x, w, bias=True)
    assert torch.equal(dx, dxb) and torch.equal(dw, dwb)
    assert torch.equal(dx, gpu.glu_linear_bwd(dy, x, w, need_dw=False)[0])
    assert torch.equal(dw, gpu.glu_linear_bwd(dy, x, w, need_dx=False)[1])
    assert torch.equal(db, gpu.glu_linear_bwd(dy, x, w, bias=True, need_dx=False, need_dw=False)[2])


@pytest.mark.parametrize("M,N,K", [(512, 1024, 512), (1021, 1000, 2056), (3000, 512, 1000), (2048, 512, 512)])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_gated(gpu, M, N, K, save):
    dh, x, w = n(M, N, seed=1), n(M, K, seed=2), (n(2 * N, K, seed=3) * K ** -0.5).to(BF16)
    _, pre, extra = gpu.glu_gated_linear(x, w, save=save)
    both = gpu.glu_gated_linear_bwd(dh, x, w, pre, extra)
    assert torch.equal(both[0], gpu.glu_gated_linear_bwd(dh, x, w, pre, extra, need_dw=False)[0])
    assert torch.equal(both[1], gpu.glu_gated_linear_bwd(dh, x, w, pre, extra, need_dx=False)[1])

"""The largest tiles of the products at every count of steps around their loops' beginnings and ends, on
small integers: every sum is exact in FP32, so the outputs are the exact results rounded once."""
import pytest
import torch

import gated_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def ints(*shape, seed=0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)


def exact(a, b):
    """a b^T of small integers: exact in FP32 in any order."""
    return a.to(F32) @ b.to(F32).t()


# 256 x 256 tiles are taken for [4096, 4096] beyond 640 elements of the sum
SUMS = [640, 648, 696, 704, 712, 768, 776, 832, 888, 896, 960, 1032]


@pytest.mark.parametrize("K", SUMS)
def test_linear(gpu, K):
    a, b = ints(4096, K, seed=K), ints(4096, K, seed=K + 1)
    assert torch.equal(gpu.glu_linear(a, b), exact(a, b).to(BF16))
    at, bt = a.t().contiguous(), b.t().contiguous()
    dx, _, _ = gpu.glu_linear_bwd(a, a.new_empty(4096, 4096), bt, need_dw=False)
    assert torch.equal(dx, exact(a, b).to(BF16))
    _, dw, _ = gpu.glu_linear_bwd(at, bt, a.new_empty(4096, 4096), need_dx=False)
    assert torch.equal(dw, exact(a, b).to(BF16))


# both gradients in one launch, of either tile size, their tiles not a multiple of 8 and ending anywhere, sums of a
# few elements to thirty-two steps; the last two take a launch each
@pytest.mark.parametrize("M,N,K", [(8, 8, 8), (1, 64, 128), (40, 1000, 264), (129, 72, 1032), (500, 520, 640), (1000, 712, 904),
                                   (1021, 1000, 2056), (1021, 2000, 2056), (704, 704, 2800), (2048, 1024, 1024), (2000, 2000, 2000),
                                   (4096, 512, 512), (300, 4096, 512)])
def test_both_gradients(gpu, M, N, K):
    dy, x, w = ints(M, N, seed=1), ints(M, K, seed=2), ints(N, K, seed=3)
    db = dy.to(F32).sum(0).to(BF16)
    dx, dw, got = gpu.glu_linear_bwd(dy, x, w, bias=True)
    assert torch.equal(dx, exact(dy, w.t()).to(BF16)) and torch.equal(dw, exact(dy.t(), x.t()).to(BF16))
    assert torch.equal(got, db)
    one, _, _ = gpu.glu_linear_bwd(dy, x, w, need_dw=False)
    _, other, _ = gpu.glu_linear_bwd(dy, x, w, need_dx=False)
    assert torch.equal(dx, one) and torch.equal(dw, other)


@pytest.mark.parametrize("K", SUMS)
@pytest.mark.parametrize("layout", ["split", "paired"])
def test_gated(gpu, K, layout):
    x, w = ints(4096, K, seed=K), ints(4096, K, seed=K + 1)
    _, pre, extra = gpu.glu_gated_linear(x, w, w_layout=layout, save="bf16")
    assert exact(x, w).abs().max() < 4096                  # within the 12 bits that are kept
    g, u = ref.halves(exact(x, w), layout, 1)
    kg, ku = ref.widened(pre, extra, 2048)
    assert torch.equal(kg.to(F32), g) and torch.equal(ku.to(F32), u)


@pytest.mark.parametrize("after", [0, 300])
def test_groups(gpu, after):
    counts = [1, 64, 65, 0, 128, 129, 193, 257, 3000, 2999, 3001, 2944, 3008, 4000, 2000, 5000]
    M, N, K = sum(counts) + after, 2048, 2048
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    x, w, dy = ints(M, K), ints(16, N, K, seed=1), ints(M, N, seed=2)
    y = gpu.glu_linear(x, w, offsets=off)
    dx, dw, _ = gpu.glu_linear_bwd(dy, x, w, offsets=off)
    for e, n in enumerate(counts):
        r = slice(int(off[e]), int(off[e]) + n)
        assert torch.equal(y[r], exact(x[r], w[e]).to(BF16))
        assert torch.equal(dx[r], exact(dy[r], w[e].t()).to(BF16))
        assert torch.equal(dw[e], exact(dy[r].t(), x[r].t()).to(BF16))
    assert (y[M - after:] == 0).all() and (dx[M - after:] == 0).all()


@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 272, 384, 496, 512, 528, 640, 768, 784, 1024])
@pytest.mark.parametrize("w_scales", ["block", "row"])
def test_8_bit(gpu, K, w_scales):
    """256 x 256 tiles are taken for [4096, 4096] whatever the sum's length."""
    M = N = 4096
    blocks = (K + 127) // 128
    x, w = ints(M, K, seed=K), ints(N, K, seed=K + 1)
    code = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(K)
    power = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").to(F32).exp2()  # noqa: E731
    xs, ws = power(blocks, M), power(*((N // 128, blocks) if w_scales == "block" else (blocks, N)))
    wide = (ws.repeat_interleave(128, 0) if w_scales == "block" else ws.t()).repeat_interleave(128, 1)[:, :K]
    y = gpu.glu_linear_fp8(code(x), xs, code(w), ws, w_scales=w_scales)
    assert torch.equal(y, exact(x.to(F32) * xs.t().repeat_interleave(128, 1)[:, :K], w.to(F32) * wide).to(BF16))

"""The gated projections and the 8-bit products on the tiles that large calls take, 256 x 256 and 256 x 128: groups
that end inside a tile, rows of no group before and after them, columns that end inside a tile, biases and codes.
test_product_plans_host.py holds each shape to the kernel named beside it."""
import pytest
import torch

import test_gpu_fp8 as fp8
import test_gpu_gated as gated

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")

# rows of each group, rows before the first and after the last, N, K, kernel
GATED_GROUPS = [([1300, 1, 0, 900, 257, 1700], 40, 1002, 776, 776, "256x256"),
                ([64, 1001, 0, 1500, 129, 3, 900], 3, 400, 776, 520, "256x128")]
GATED = [(3100, 1288, 776, "256x256"), (3000, 1032, 520, "256x128")]
FP8_GROUPS = [([1200, 1, 0, 900, 257, 1700, 300], 40, 602, 2056, 1040, "256x256"),
              ([64, 1001, 0, 1500, 129, 3, 900], 3, 400, 1544, 1040, "256x128")]
FP8 = [(4100, 2312, 528, "256x256"), (3001, 1288, 1040, "256x128"), (4000, 2008, 528, "256x128")]


def offsets_of(counts, before):
    return before + torch.tensor([0] + counts, device="cuda").cumsum(0).int()


@pytest.mark.parametrize("counts,before,after,N,K,kernel", GATED_GROUPS, ids=[c[-1] for c in GATED_GROUPS])
@pytest.mark.parametrize("layout", ["split", "paired"])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
@pytest.mark.parametrize("act", ["swiglu", "geglu_erf"])
def test_gated_groups(gpu, counts, before, after, N, K, kernel, layout, save, act):
    M = before + sum(counts) + after
    t = gated.draw(M, N, K, groups=len(counts), seed=M)
    for r in (slice(0, before), slice(M - after, M)):   # rows of no group: whatever they hold, zeros come out
        t["x"][r], t["dh"][r] = NAN, INF
    out = gated.check(gpu, t, act, layout, save, offsets_of(counts, before))
    h, pre, dx, again = out[0], out[2], out[4], out[7]
    for r in (slice(0, before), slice(M - after, M)):
        assert not any(v[r].any() for v in (h, pre, dx, again))


@pytest.mark.parametrize("M,N,K,kernel", GATED)
@pytest.mark.parametrize("layout", ["split", "paired"])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_gated(gpu, M, N, K, kernel, layout, save):
    gated.check(gpu, gated.draw(M, N, K, seed=N), "geglu", layout, save)


@pytest.mark.parametrize("counts,before,after,N,K,kernel", FP8_GROUPS, ids=[c[-1] for c in FP8_GROUPS])
@pytest.mark.parametrize("w_scales", ["block", "row"])
def test_fp8_groups(gpu, counts, before, after, N, K, kernel, w_scales):
    M = before + sum(counts) + after
    t = fp8.operands(M, N, K, w_scales, len(counts), seed=M)
    for r in (slice(0, before), slice(M - after, M)):
        t["xq"][r], t["xs"][:, r], t["residual"][r] = 0x7f, NAN, NAN
    y = fp8.check_product(gpu, t, w_scales, offsets_of(counts, before))
    assert not y[:before].any() and not y[M - after:].any()


@pytest.mark.parametrize("M,N,K,kernel", FP8)
@pytest.mark.parametrize("w_scales", ["block", "row"])
def test_fp8(gpu, M, N, K, kernel, w_scales):
    fp8.check_product(gpu, fp8.operands(M, N, K, w_scales, seed=N), w_scales)

"""Which gradients the torch ops around the GLU give, and which not."""
import pytest
import torch

import glu_activation_microscaling_amd.torch_ops  # noqa: F401

pytestmark = pytest.mark.gpu
ops = torch.ops.glu_mx
BF16 = torch.bfloat16


def n(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("first,last", [(0, 50), (0, 40), (4, 50), (4, 40), (-3, 70), (20, 20), (60, 70)])
def test_the_residual_s_gradient_is_zero_in_rows_of_no_group(gpu, act, first, last):
    """There y is zero and holds no residual, so whatever dy is there, NaN included, goes nowhere."""
    x, w, res = n(50, 64), n(3, 72, 64, seed=1), n(50, 72, seed=2).requires_grad_(True)
    middle = (first + last) // 2
    off = torch.tensor([first, middle, middle, last], dtype=torch.int32, device="cuda")
    inside = torch.zeros(50, dtype=torch.bool, device="cuda")
    inside[max(first, 0):max(last, 0)] = True
    dy = n(50, 72, seed=3)
    dy[~inside] = float("nan")
    y, _ = ops.linear(x, w, None, res, off, act)
    (got,) = torch.autograd.grad(y, res, dy)
    assert torch.equal(got, torch.where(inside.unsqueeze(1), dy, torch.zeros_like(dy)))

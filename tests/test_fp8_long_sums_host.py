"""W's gradient of an 8-bit linear layer sums over the rows of x: as many rows as the product takes, and a
call of more is refused before its forward (no GPU)."""
import ctypes

import pytest
import torch

import glu_activation_microscaling_amd as glu
import glu_activation_microscaling_amd.torch_ops  # noqa: F401
from test_abi_host import OK, SHAPE
from test_gated_host import product, setup_module  # noqa: F401

ops = torch.ops.glu_mx


def test_the_gradients_sum_is_as_long_as_the_rows():
    long = dict(M=72, N=64, ld_y=64, ld_res=64, mode=1, bytes=1 << 30)
    assert product(K=1048592, **long) == OK and product(K=1 << 22, **long) == OK
    assert product(K=(1 << 22) + 16, **long) == SHAPE and product(K=1048592, **{**long, "mode": 0}) == SHAPE
    work = glu.lib().glu_linear_fp8_work_bytes
    assert work(72, 64, 1 << 22, 1, 0) >= 0 and work(72, 64, (1 << 22) + 16, 1, 0) == -1
    assert ctypes.c_int64(work(1, 8, 1048592, 1, 0)).value >= 0


def rows(M, grad):
    return torch.empty(M, 16, dtype=torch.bfloat16, device="meta").requires_grad_(grad)


def test_a_forward_whose_gradient_cannot_be_formed_is_refused():
    most, w = 1 << 22, torch.empty(8, 16, dtype=torch.bfloat16, device="meta")
    assert ops.linear_fp8(rows(most, True), w.clone().requires_grad_(True))[0].shape == (most, 8)
    with pytest.raises(ValueError, match="rows for the gradient of w"):
        ops.linear_fp8(rows(most + 16, False), w.clone().requires_grad_(True))
    # without that gradient any number of rows
    assert ops.linear_fp8(rows(most + 16, True), w)[0].shape == (most + 16, 8)
    with torch.no_grad():
        assert ops.linear_fp8(rows(most + 16, True), w.clone().requires_grad_(True))[0].shape == (most + 16, 8)

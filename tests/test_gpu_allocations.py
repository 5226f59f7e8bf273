"""What the gated, checkpointed and 8-bit entry points allocate: seen by dispatch modes, and filled where
deterministic mode fills memory that nothing has written."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from glu_activation_microscaling_amd import ffn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def n(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def calls(gpu):
    x, w, dh = n(300, 136), n(144, 136, seed=1), n(300, 72, seed=2)
    h, pre, extra = gpu.glu_gated_linear(x, w, save="mxfp8")
    _, q, s = gpu.glu_fwd_ckpt(h, dh)
    qr, _, sr, _ = gpu.glu_quant_fp8(x)
    wq, ws, _, _ = gpu.glu_quant_fp8_weight(w)
    return [lambda: [gpu.glu_gated_linear(x, w)], lambda: gpu.glu_gated_linear(x, w, save="bf16"),
            lambda: gpu.glu_gated_linear_bwd(dh, x, w, pre, extra, bias=True, need_h=True), lambda: gpu.glu_fwd_ckpt(h, dh),
            lambda: gpu.glu_bwd_ckpt(q, s, dh, need_h=True), lambda: gpu.glu_quant_fp8(x, colwise=True),
            lambda: gpu.glu_fwd_fp8(h, dh, colwise=True), lambda: gpu.glu_quant_fp8_weight(w, transpose=True),
            lambda: [gpu.glu_linear_fp8(qr, sr, wq, ws)]]


class Allocations(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in func.__name__:
            self.made.add(out.data_ptr())
        return out


def test_dispatch_modes_see_every_output(gpu):
    for i, f in enumerate(calls(gpu)):
        with Allocations() as seen:
            out = f()
        assert out and all(t.numel() == 0 or t.data_ptr() in seen.made for t in out), i


def test_deterministic_mode_fills_what_is_allocated(gpu):
    assert torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    try:
        assert torch.isnan(ffn._allocator(n(8))((64, 40), BF16)).all() and torch.isnan(ffn._contiguous((2, 3, 8), BF16)).all()
    finally:
        torch.use_deterministic_algorithms(False)

"""Outputs and scratch memory are allocated where torch sees it: by dispatch modes (no GPU)."""
import torch
from torch._subclasses.fake_tensor import FakeTensor, FakeTensorMode

from glu_activation_microscaling_amd import ffn


def test_dispatch_modes_see_the_allocation(monkeypatch):
    monkeypatch.setattr(ffn, "_device", lambda: 0)
    with FakeTensorMode():
        ref = torch.empty(4, dtype=torch.bfloat16, device="cuda:0")
        for new in (ffn._allocator(ref), ffn._contiguous):
            for shape in ((0,), (5,), (3, 8), (2, 3, 4), (0, 7)):
                t = new(shape, torch.uint8)
                assert isinstance(t, FakeTensor) and t.device.type == "cuda" and t.is_contiguous()
                assert tuple(t.shape) == shape and t.dtype == torch.uint8

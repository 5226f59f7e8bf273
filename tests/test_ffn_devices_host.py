"""The linear products on operands of another device than the current one: the call is made on theirs (no GPU)."""
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import glu_activation_microscaling_amd as glu
from glu_activation_microscaling_amd import ffn


def test_linear_calls_are_made_on_their_operands_device(monkeypatch):
    log = []

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            log.append(("enter", self.i))

        def __exit__(self, *_):
            log.append(("exit", self.i))

    monkeypatch.setattr(ffn, "_device", lambda: 0)
    monkeypatch.setattr(ffn, "_raw_stream", lambda i: ("stream", i))
    monkeypatch.setattr(ffn, "_ptr", lambda t: None)
    monkeypatch.setattr(ffn, "_call", lambda name, *args: log.append((name, args[-1])))
    monkeypatch.setattr(torch.cuda, "device", Device)
    with FakeTensorMode():
        x, w, dy = (torch.empty(s, dtype=torch.bfloat16, device="cuda:1") for s in ((40, 64), (72, 64), (40, 72)))
        glu.glu_linear(x, w)
        glu.glu_linear_bwd(dy, x, w, bias=True)
    assert log == [("enter", 1), ("glu_linear", ("stream", 1)), ("exit", 1),
                   ("enter", 1), ("glu_linear_bwd", ("stream", 1)), ("exit", 1)]

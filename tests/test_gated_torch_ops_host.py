"""The gated, checkpointed and 8-bit torch ops without a GPU: shapes of the fake implementations, and
gradients that route to the backward ops."""
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

import glu_activation_microscaling_amd.torch_ops  # noqa: F401

ops = torch.ops.glu_mx


def b(*shape, dtype=torch.bfloat16, device="cuda"):
    return torch.empty(shape, dtype=dtype, device=device)


def shapes(ts):
    return [tuple(t.shape) for t in ts]


def test_fake_shapes():
    u8, f32 = torch.uint8, torch.float32
    with FakeTensorMode():
        x, w = b(40, 64), b(144, 64)
        h = ops.gated_linear(x, w)
        assert shapes(h) == [(40, 72), (40, 144), (40, 72)] and [t.dtype for t in h] == [torch.bfloat16, torch.bfloat16, u8]
        h = ops.gated_linear(x, w, None, None, "geglu", "paired", "mxfp8")
        assert shapes(h) == [(40, 72), (40, 144), (40, 6)] and h[1].dtype == u8
        assert shapes(ops.gated_linear(x, w, None, None, "geglu", "paired", "none")) == [(40, 72), (0,), (0,)]
        off = b(4, dtype=torch.int32)
        h = ops.gated_linear(x, b(3, 144, 64), b(3, 144), off)
        g = ops.gated_linear_backward(h[0], x, b(3, 144, 64), h[1], h[2], off, "swiglu", "split", True)
        assert shapes(g) == [(40, 64), (3, 144, 64), (3, 144)]
        c = ops.glu_ckpt(b(40, 72), b(40, 72))
        assert shapes(c) == [(40, 72), (40, 144), (40, 6)]
        assert shapes(ops.glu_ckpt(b(40, 144), b(0), "swiglu", "paired")) == shapes(c)
        assert shapes(ops.glu_ckpt_backward(c[1], c[2], c[0], "swiglu", "split", True)) == [(40, 144), (40, 72)]
        y = ops.feed_forward(x, w, b(56, 72))
        assert shapes(y) == [(40, 56), (40, 144), (40, 6)]
        g = ops.feed_forward_backward(y[0], x, w, b(56, 72), y[1], y[2], None, "swiglu", "split", True, False)
        assert shapes(g) == [(40, 64), (144, 64), (56, 72), (144,), (0,)]
        q = ops.quant_fp8(b(40, 136), True, True)
        assert shapes(q) == [(40, 144), (136, 48), (2, 40), (1, 136)] and [t.dtype for t in q] == [u8, u8, f32, f32]
        assert shapes(ops.glu_fp8(b(40, 272), b(0), "swiglu", "paired")) == [(40, 144), (0,), (2, 40), (0,)]
        wq = ops.quant_fp8_weight(b(3, 136, 264), True)
        assert shapes(wq) == [(3, 136, 272), (3, 2, 3), (3, 264, 144), (3, 3, 2)]
        y = ops.product_fp8(q[0], q[2], b(200, 144, dtype=u8), b(2, 2, dtype=f32))
        assert y.shape == (40, 200) and y.dtype == torch.bfloat16
        y = ops.linear_fp8(x, w)
        assert shapes(y) == [(40, 144), (64, 48), (1, 64), (64, 144), (1, 2)]
        assert shapes(ops.linear_fp8_backward(y[0], *y[1:], True, True, True)) == [(40, 64), (144, 64), (144,)]


def test_autograd_routes_to_the_backward_ops():
    def f(x, w13, w2, gate, up):
        x, w13, w2, gate, up = (t.detach().requires_grad_(True) for t in (x, w13, w2, gate, up))
        h, _, _ = ops.gated_linear(x, w13)
        y, _, _ = ops.feed_forward(x, w13, w2)
        z = ops.linear_fp8(h, w2)[0]
        c = ops.glu_ckpt(gate, up)[0]
        return torch.autograd.grad(y.sum() + z.sum() + c.sum(), (x, w13, w2, gate, up))

    m = dict(device="meta")
    gm = make_fx(f)(b(8, 64, **m), b(48, 64, **m), b(32, 24, **m), b(8, 24, **m), b(8, 24, **m))
    names = [str(t.target) for t in gm.graph.nodes if t.op == "call_function"]
    for op in ("gated_linear_backward", "feed_forward_backward", "linear_fp8_backward", "glu_ckpt_backward"):
        assert any("glu_mx." + op in s for s in names), op


def test_side_outputs_have_no_gradient():
    x, w = (b(*s, device="meta").requires_grad_(True) for s in ((8, 64), (48, 64)))
    for out in (ops.gated_linear(x, w), ops.feed_forward(x, w, b(64, 24, device="meta")),
                ops.linear_fp8(x, b(48, 64, device="meta")), ops.glu_ckpt(x, x)):
        assert out[0].requires_grad and not any(t.requires_grad for t in out[1:])

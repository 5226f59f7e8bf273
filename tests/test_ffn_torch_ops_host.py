"""The operators around the GLU as torch ops without a GPU: shapes of the fake implementations, and
gradients that route to the backward ops."""
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

import glu_activation_microscaling_amd.torch_ops  # noqa: F401

ops = torch.ops.glu_mx


def b(*shape, dtype=torch.bfloat16, device="cuda"):
    return torch.empty(shape, dtype=dtype, device=device)


def test_fake_shapes():
    with FakeTensorMode():
        x, y, w = b(40, 64, dtype=torch.float32), b(40, 64), b(64)
        xo, h, st = ops.block_norm(x, y, w, w, w, w, True)
        assert xo.shape == h.shape == (40, 64) and xo.dtype == torch.float32 and h.dtype == torch.bfloat16
        assert st.shape == (40, 4) and ops.block_norm(x)[0].numel() == 0
        g = ops.block_norm_backward(x, y, st, xo, h, w, w, None, w, True, 1.0, "rms")
        assert [t.shape for t in g] == [(40, 64), (40, 64), (64,), (64,), (64,), (0,)]
        off = b(4, dtype=torch.int32)
        yy, pre = ops.linear(y, b(3, 24, 64), None, None, off, "silu")
        assert yy.shape == pre.shape == (40, 24) and pre.dtype == torch.float16
        assert ops.linear(y, b(24, 64))[1].numel() == 0
        g = ops.linear_backward(yy, y, b(3, 24, 64), pre, off, "silu", True)
        assert [t.shape for t in g] == [(40, 64), (3, 24, 64), (3, 24)]
        rows, offsets = ops.moe_sort(b(40, 2, dtype=torch.int64), 8)
        assert rows.shape == (40, 2) and offsets.shape == (9,) and rows.dtype == torch.int32
        xs = ops.moe_permute(y, rows, offsets)
        assert xs.shape == (80, 64) and ops.moe_combine(xs, rows, offsets).shape == (40, 64)
        g = ops.moe_combine_backward(y, xs, rows, b(40, 2, dtype=torch.float32), offsets)
        assert [t.shape for t in g] == [(80, 64), (40, 2)]


def test_autograd_routes_to_the_backward_ops():
    def f(x, y, w, wt, ids):
        x, y, w, wt = (t.detach().requires_grad_(True) for t in (x, y, w, wt))
        xo, h, _ = ops.block_norm(x, y, w, w, None, None)
        rows, off = ops.moe_sort(ids, 2)
        xs = ops.moe_permute(h, rows, off)
        a, _ = ops.linear(xs, wt, None, None, off, "gelu")
        out = ops.moe_combine(a, rows, off, torch.ones(rows.shape, device="meta"))
        return torch.autograd.grad(xo.sum() + out.sum(), (x, y, w, wt))

    m = dict(device="meta")
    gm = make_fx(f)(b(8, 64, **m), b(8, 64, **m), b(64, **m), b(2, 64, 64, **m), b(8, 2, dtype=torch.int32, **m))
    names = [str(t.target) for t in gm.graph.nodes if t.op == "call_function"]
    for op in ("block_norm_backward", "linear_backward", "moe_combine_backward", "moe_combine.default"):
        assert any("glu_mx." + op in s for s in names), op


def test_side_outputs_have_no_gradient():
    """stats and pre serve the backward: a loss on them is refused by autograd, not given zeros."""
    x, w = (b(*s, device="meta").requires_grad_(True) for s in ((8, 64), (24, 64)))
    y = b(8, 64, device="meta")
    xo, h, stats = ops.block_norm(x, y)
    assert xo.requires_grad and h.requires_grad and not stats.requires_grad
    for act in ("none", "silu"):
        out, pre = ops.linear(x, w, None, None, None, act)
        assert out.requires_grad and not pre.requires_grad


def test_linear_s_backward_is_asked_for_what_is_wanted():
    m = dict(device="meta")

    def wanted(*names, act="silu"):
        """(bias, need_dx, need_dw) of the backward op's call when these operands want gradients; None: no call."""
        def f(x, w, bias, residual):
            t = dict(x=x, w=w, bias=bias, residual=residual)
            t.update({k: t[k].detach().requires_grad_(True) for k in names})
            y, _ = ops.linear(t["x"], t["w"], t["bias"], t["residual"], None, act)
            return torch.autograd.grad(y.sum(), [t[k] for k in names])

        gm = make_fx(f)(b(8, 64, **m), b(24, 64, **m), b(24, **m), b(8, 24, **m))
        calls = [n.args + (True,) * (9 - len(n.args)) for n in gm.graph.nodes if "linear_backward" in str(n.target)]
        assert len(calls) <= 1
        return calls[0][6:] if calls else None

    assert wanted("x", "w", "bias") == (True, True, True) and wanted("x", "residual") == (False, True, False)
    assert wanted("w") == (False, False, True) and wanted("bias") == (True, False, False)
    assert wanted("residual") is None and wanted("residual", act="none") is None

    # arguments by name and left out
    x, w, r = (b(*s, **m).requires_grad_(True) for s in ((8, 64), (24, 64), (8, 24)))
    for y, given in ((ops.linear(x, w), False), (ops.linear(x, w, act="silu"), False), (ops.linear(x, w, None, r), True),
                     (ops.linear(x, w, residual=r, act="silu"), True)):
        g = torch.autograd.grad(y[0].sum(), (x, w, r), allow_unused=True)
        assert [t is not None for t in g] == [True, True, given]
    y = ops.linear(x.detach(), w=w.detach(), residual=r)[0]
    assert torch.autograd.grad(y.sum(), r)[0].shape == r.shape

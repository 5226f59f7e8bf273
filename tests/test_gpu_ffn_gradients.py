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


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_gradients_of_linear_by_ones_and_twos(gpu, act):
    """A gradient has the same bits whichever others are wanted with it."""
    args = dict(x=n(50, 64), w=n(72, 64, seed=1), bias=n(72, seed=2), residual=n(50, 72, seed=3))
    dy = n(50, 72, seed=4)

    def grads(*names):
        t = {k: v.clone().requires_grad_(k in names) for k, v in args.items()}
        y, _ = ops.linear(t["x"], t["w"], t["bias"], t["residual"], None, act)
        return dict(zip(names, torch.autograd.grad(y, [t[k] for k in names], dy)))

    full = grads(*args)
    for names in (("x",), ("w",), ("bias",), ("residual",), ("x", "bias"), ("w", "residual"), ("x", "w")):
        for k, g in grads(*names).items():
            assert torch.equal(g, full[k]), (names, k)


def test_the_residual_alone_needs_no_pre_activation(gpu):
    x, w, res, dy = n(50, 64), n(72, 64, seed=1), n(50, 72, seed=2).requires_grad_(True), n(50, 72, seed=3)
    y, pre = ops.linear(x, w, None, res, None, "silu", False)
    assert pre.numel() == 0
    assert torch.equal(torch.autograd.grad(y, res, dy)[0], dy)
    y, _ = ops.linear(x, w, n(72, seed=4).requires_grad_(True), res, None, "silu", False)
    with pytest.raises(RuntimeError):
        y.sum().backward()


@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradients_of_no_rows(gpu, act):
    """A batch without tokens: the gradient of a sum over no rows is an expanded tensor.  Parameters get
    zeros, the rest is empty."""
    def leaf(*shape, dtype=BF16):
        return torch.ones(shape, device="cuda", dtype=dtype).requires_grad_(True)

    x, y, w = leaf(0, 64), leaf(0, 64), leaf(64)
    xo, h, _ = ops.block_norm(x, y, w, w, w, w, True)
    for t, g in zip((x, y, w), torch.autograd.grad(xo.sum() + h.sum(), (x, y, w))):
        assert g.shape == t.shape and (g == 0).all()
    wt, b, res = leaf(3, 72, 64), leaf(3, 72), leaf(0, 72)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    for args in ((x, wt, b, res, off), (x, leaf(72, 64), leaf(72), res, None)):
        out, _ = ops.linear(*args, act)
        for t, g in zip(args, torch.autograd.grad(out.sum(), args[:4])):
            assert g.shape == t.shape and (g == 0).all()
    rows, offsets = ops.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    ys, wts = leaf(0, 64), leaf(0, 2, dtype=torch.float32)
    for out in (ops.moe_permute(x, rows, offsets), ops.moe_combine(ys, rows, offsets, wts, y),
                ops.moe_combine(ys, rows, offsets)):
        for g in torch.autograd.grad(out.sum(), (x, y, ys, wts), allow_unused=True):
            assert g is None or g.numel() == 0


def test_gradients_that_start_off_a_16_byte_boundary(gpu):
    """The gradient of one part of a concatenation is a view that starts where the part does: at widths that
    are no multiple of 8, anywhere.  It gives the bits of the same gradient on a boundary."""
    H = 101
    x, y, w = (t.requires_grad_(True) for t in (n(6, H), n(6, H, seed=1), n(H, seed=2)))
    ids = torch.randint(0, 3, (6, 2), device="cuda", dtype=torch.int32)
    rows, offsets = ops.moe_sort(ids, 3)
    wts = torch.rand(6, 2, device="cuda").requires_grad_(True)
    ys = n(12, H, seed=3).requires_grad_(True)
    for make, leaves in ((lambda: ops.block_norm(x, y, w, w, w, w, True)[0], (x, y, w)),
                         (lambda: ops.block_norm(x, y, w, w, w, w, True)[1], (x, y, w)),
                         (lambda: ops.moe_permute(x, rows, offsets), (x,)),
                         (lambda: ops.moe_combine(ys, rows, offsets, wts, y), (ys, wts, y)),
                         (lambda: ops.moe_combine(ys, rows, offsets), (ys,))):
        t = make()
        d = n(t.shape[0] + 1, H, seed=4)
        want = torch.autograd.grad(t, leaves, d[1:].clone())
        t = torch.cat([n(1, H), make()])
        for a, b in zip(torch.autograd.grad(t, leaves, d), want):
            assert torch.equal(a, b)
    wt, res = n(40, 72, seed=5).requires_grad_(True), n(6, 40, seed=6).requires_grad_(True)
    t = ops.linear(n(6, 72), wt, None, res, None, "silu")[0]
    d = n(1 + 240, seed=7)
    want = torch.autograd.grad(t, (wt, res), d[1:].reshape(6, 40).clone())
    t = torch.cat([n(1), ops.linear(n(6, 72), wt, None, res, None, "silu")[0].flatten()])
    for a, b in zip(torch.autograd.grad(t, (wt, res), d), want):
        assert torch.equal(a, b)

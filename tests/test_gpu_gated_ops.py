"""The gated projections, checkpoints and 8-bit linear layers as torch ops: forward and gradients equal to
the entry points composed by hand, compiled whole, and used together in a block."""
import os
import sys

import pytest
import torch

import glu_activation_microscaling_amd.torch_ops  # noqa: F401
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import feed_forward as example  # noqa: E402

pytestmark = pytest.mark.gpu
ops = torch.ops.glu_mx
BF16 = torch.bfloat16


def n(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def leaf(*shape, **kw):
    return n(*shape, **kw).requires_grad_(True)


OFFSETS = [None, [3, 20, 20, 70]]


@pytest.mark.parametrize("offsets", OFFSETS, ids=["dense", "groups"])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
@pytest.mark.parametrize("layout", ["split", "paired"])
def test_gated_linear(gpu, offsets, save, layout):
    lead = () if offsets is None else (3,)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x, w, b, dh = leaf(75, 136), leaf(*lead, 144, 136, seed=1, scale=0.1), leaf(*lead, 144, seed=2), n(75, 72, seed=3)
    h, pre, extra = ops.gated_linear(x, w, b, off, "geglu", layout, save)
    assert h.requires_grad and not pre.requires_grad and not extra.requires_grad
    got = torch.autograd.grad(h, (x, w, b), dh)
    p = dict(act="geglu", w_layout=layout, offsets=off)
    hh, pp, ee = gpu.glu_gated_linear(x.detach(), w.detach(), b.detach(), save=save, **p)
    want = gpu.glu_gated_linear_bwd(dh, x.detach(), w.detach(), pp, ee, bias=True, **p)
    assert torch.equal(h, hh) and all(torch.equal(u, v) for u, v in zip(got, want))
    # some of the gradients alone, and a gradient that starts off a 16-byte boundary
    only = torch.autograd.grad(ops.gated_linear(x.detach(), w, None, off, "geglu", layout, save)[0], w, dh)[0]
    assert only.shape == w.shape
    wide = n(75, 76, seed=3)
    off_boundary = torch.autograd.grad(ops.gated_linear(x, w, b, off, "geglu", layout, save)[0], x, wide[:, 4:])[0]
    again = torch.autograd.grad(ops.gated_linear(x, w, b, off, "geglu", layout, save)[0], x, wide[:, 4:].clone())[0]
    assert torch.equal(off_boundary, again)


def test_what_was_not_kept_has_no_gradient(gpu):
    x, w = leaf(8, 64), leaf(48, 64)
    h, pre, extra = ops.gated_linear(x, w, None, None, "swiglu", "split", "none")
    assert pre.numel() == 0 and extra.numel() == 0
    with pytest.raises(RuntimeError, match="not kept"):
        torch.autograd.grad(h.sum(), x)
    y, _, _ = ops.feed_forward(x, w, leaf(64, 24, seed=2), None, None, None, "swiglu", "split", "none")
    with pytest.raises(RuntimeError, match="not kept"):
        torch.autograd.grad(y.sum(), x)


@pytest.mark.parametrize("layout", ["split", "paired"])
def test_glu_ckpt(gpu, layout):
    g, u, dh = n(40, 72), n(40, 72, seed=1), n(40, 72, seed=2)
    if layout == "split":
        leaves = [g.requires_grad_(True), u.requires_grad_(True)]
        args = leaves
    else:
        leaves = [torch.stack([g, u], 2).flatten(1).requires_grad_(True)]
        args = [leaves[0], g.new_empty((0,))]
    h, q, s = ops.glu_ckpt(*args, "geglu", layout)
    got = torch.autograd.grad(h, leaves, dh)
    d, _ = gpu.glu_bwd_ckpt(q, s, dh, act="geglu", layout=layout)
    assert torch.equal(torch.cat(got, 1), d) and torch.equal(h, gpu.glu_fwd(g.detach(), u.detach(), act="geglu"))
    # nothing but the codes and their scales is kept for the backward
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t.dtype) or t, lambda t: t):
        ops.glu_ckpt(*args, "geglu", layout)
    assert kept == [torch.uint8, torch.uint8]


@pytest.mark.parametrize("offsets", OFFSETS, ids=["dense", "groups"])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_feed_forward(gpu, offsets, save):
    lead = () if offsets is None else (3,)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x, w13, w2 = leaf(75, 136), leaf(*lead, 144, 136, seed=1, scale=0.1), leaf(*lead, 136, 72, seed=2, scale=0.1)
    b13, b2, dy = leaf(*lead, 144, seed=3), leaf(*lead, 136, seed=4), n(75, 136, seed=5)
    y, pre, extra = ops.feed_forward(x, w13, w2, b13, b2, off, "swiglu", "split", save)
    got = torch.autograd.grad(y, (x, w13, w2, b13, b2), dy)
    X, W13, W2, B13, B2 = (t.detach() for t in (x, w13, w2, b13, b2))
    h, p, e = gpu.glu_gated_linear(X, W13, B13, offsets=off, save=save)
    assert torch.equal(y, gpu.glu_linear(h, W2, B2, offsets=off)) and torch.equal(pre, p) and torch.equal(extra, e)
    dh, _, _ = gpu.glu_linear_bwd(dy, h, W2, offsets=off)
    dx, dw13, db13, hk = gpu.glu_gated_linear_bwd(dh, X, W13, p, e, offsets=off, bias=True, need_h=True)
    _, dw2, db2 = gpu.glu_linear_bwd(dy, hk, W2, offsets=off, bias=True)
    for a, b in zip(got, (dx, dw13, dw2, db13, db2)):
        assert torch.equal(a, b)
    # without biases, and only some of the leaves
    y, _, _ = ops.feed_forward(x.detach(), W13, w2, None, None, off, "swiglu", "split", save)
    assert torch.autograd.grad(y, w2, dy)[0].shape == w2.shape


def test_linear_fp8(gpu):
    x, w, b, r, dy = leaf(75, 136), leaf(200, 136, seed=1, scale=0.1), leaf(200, seed=2), leaf(75, 200, seed=3), n(75, 200, seed=4)
    y = ops.linear_fp8(x, w, b, r)[0]
    dx, dw, db, dr = torch.autograd.grad(y, (x, w, b, r), dy)
    xr, xc, sxr, sxc = gpu.glu_quant_fp8(x.detach(), colwise=True)
    wq, ws, wt, wts = gpu.glu_quant_fp8_weight(w.detach(), transpose=True)
    qr, qc, sr, sc = gpu.glu_quant_fp8(dy, colwise=True)
    assert torch.equal(y, gpu.glu_linear_fp8(xr, sxr, wq, ws, b.detach(), r.detach()))
    assert torch.equal(dx, gpu.glu_linear_fp8(qr, sr, wt, wts)) and torch.equal(dr, dy)
    assert torch.equal(dw, gpu.glu_linear_fp8(qc, sc, xc, sxc, w_scales="row"))
    want = dy.double().sum(0)
    assert ((db.double() - want).abs() <= 2.0 ** -8 * want.abs() + 75 * 2.0 ** -23 * dy.double().abs().sum(0)).all()
    y = ops.linear_fp8(x.detach(), w, b)[0]
    assert torch.equal(torch.autograd.grad(y, w, dy)[0], dw)


def test_opcheck(gpu):
    x, w, w2 = leaf(24, 72), leaf(80, 72, seed=1, scale=0.1), leaf(72, 40, seed=2, scale=0.1)
    off = torch.tensor([2, 10, 20], dtype=torch.int32, device="cuda")
    torch.library.opcheck(ops.gated_linear, (x, w, leaf(80, seed=3), None, "swiglu", "paired", "bf16"))
    torch.library.opcheck(ops.gated_linear, (x, leaf(2, 80, 72, seed=1), None, off, "geglu", "split", "mxfp8"))
    torch.library.opcheck(ops.glu_ckpt, (leaf(24, 40), leaf(24, 40, seed=1), "relu2", "split"))
    torch.library.opcheck(ops.feed_forward, (x, w, w2, None, None, None, "swiglu", "split", "mxfp8"))
    torch.library.opcheck(ops.linear_fp8, (x, w, leaf(80, seed=3), leaf(24, 80, seed=4)))
    torch.library.opcheck(ops.quant_fp8, (n(24, 72), True, True))
    torch.library.opcheck(ops.glu_fp8, (n(24, 72), n(24, 72, seed=1), "geglu", "split", True, True))
    torch.library.opcheck(ops.quant_fp8_weight, (n(3, 40, 72), True))
    q, _, s, _ = ops.quant_fp8(n(24, 72))
    wq, ws, _, _ = ops.quant_fp8_weight(n(40, 72), False)
    torch.library.opcheck(ops.product_fp8, (q, s, wq, ws, n(40), n(24, 40), None, "block"))


@pytest.mark.parametrize("experts,choices", [(0, 0), (6, 2)])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_a_block_of_them_compiles_whole_and_equals_eager(gpu, experts, choices, save):
    p = example.make_params(200, 328, experts)
    x, y, d = (n(150, 200, seed=i).requires_grad_(i < 2) for i in range(3))
    leaves = [x, y] + list(p.values())

    def step(x, y, p):
        return example.feed_forward(x, y, p, choices, save)

    eager = step(x, y, p)
    compiled = torch.compile(step, fullgraph=True, backend="aot_eager")(x, y, p)
    for a, b in zip(eager, compiled):
        assert torch.equal(a, b)
    grads = torch.autograd.grad(eager, leaves, [d, d])
    for a, b in zip(grads, torch.autograd.grad(compiled, leaves, [d, d])):
        assert torch.equal(a, b)
    # the block by the projections and the GLU one by one: the same function, so near in every gradient.
    # Each path rounds a handful of intermediates to BF16 (2^-8 at most), 8-bit codes to 4 bits (2^-4).
    plain = example.feed_forward(x, y, p, choices)
    near = 6 * 2.0 ** -8 + (2 * 2.0 ** -4 if save == "mxfp8" else 0.0)
    for a, b in zip((*eager, *grads), (*plain, *torch.autograd.grad(plain, leaves, [d, d]))):
        assert (a.double() - b.double()).norm() <= near * b.double().norm()


def test_the_example_runs(gpu):
    for kw in (dict(save="bf16"), dict(save="mxfp8"), dict(save="mxfp8", experts=4, choices=2)):
        losses = example.train(tokens=64, width=64, inner=72, steps=2, **kw)
        assert len(losses) == 2 and all(v == v and v < float("inf") for v in losses)


def test_no_rows(gpu):
    x, w, w2 = leaf(0, 136), leaf(144, 136, seed=1), leaf(200, 72, seed=2)
    b, r = leaf(200, seed=3), leaf(0, 200, seed=4)
    for save in ("bf16", "mxfp8"):
        h = ops.gated_linear(x, w, None, None, "swiglu", "split", save)[0]
        y = ops.feed_forward(x, w, w2, None, b, None, "swiglu", "split", save)[0]
        assert h.shape == (0, 72) and y.shape == (0, 200)
        for a, z in zip(torch.autograd.grad(h.sum() + y.sum(), (x, w, w2, b)), (x, w, w2, b)):
            assert a.shape == z.shape and (a == 0).all()
    z = ops.linear_fp8(h.detach().requires_grad_(True), w2, b, r)[0]
    for a, t in zip(torch.autograd.grad(z.sum(), (w2, b, r)), (w2, b, r)):
        assert a.shape == t.shape and (a == 0).all()
    assert ops.glu_ckpt(leaf(0, 72), leaf(0, 72))[0].shape == (0, 72)


def test_expanded_gradients_and_halves_of_one_tensor(gpu):
    """The gradient of a sum has no strides; gate and up may be the halves of one projection."""
    both, w, x = leaf(40, 144), leaf(144, 136, seed=1, scale=0.1), leaf(40, 136, seed=2)
    ones = torch.ones(40, 72, device="cuda", dtype=BF16)
    h = ops.glu_ckpt(*both.chunk(2, 1))[0]
    assert torch.equal(torch.autograd.grad(h.sum(), both)[0], torch.autograd.grad(ops.glu_ckpt(*both.chunk(2, 1))[0], both, ones)[0])
    for f in (lambda: ops.gated_linear(x, w)[0], lambda: ops.linear_fp8(x, w[:72])[0]):
        for a, b in zip(torch.autograd.grad(f().sum(), (x, w)), torch.autograd.grad(f(), (x, w), ones)):
            assert torch.equal(a, b)


def test_offsets_out_of_range_are_taken_into_it(gpu):
    x, w = n(40, 136), n(2, 144, 136, seed=1, scale=0.1)
    far = torch.tensor([-7, 20, 10 ** 9], dtype=torch.int32, device="cuda")
    near = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    dh = n(40, 72, seed=2)
    q, _, s, _ = gpu.glu_quant_fp8(x)
    wq, ws, _, _ = gpu.glu_quant_fp8_weight(w)
    for save in ("bf16", "mxfp8"):
        got, want = [], []
        for out, off in ((got, far), (want, near)):
            h, pre, extra = gpu.glu_gated_linear(x, w, offsets=off, save=save)
            out += [h, pre, extra, *gpu.glu_gated_linear_bwd(dh, x, w, pre, extra, offsets=off, bias=True, need_h=True),
                    gpu.glu_linear_fp8(q, s, wq, ws, offsets=off)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_a_captured_training_step(gpu, save):
    """Forward and backward in one graph, replayed between eager work; the leaves have no eager graph."""
    x, w13, w2 = leaf(150, 136), leaf(656, 136, seed=1, scale=0.1), leaf(136, 328, seed=2, scale=0.1)
    w8, b8, d = leaf(136, 136, seed=3, scale=0.1), leaf(136, seed=4), n(150, 136, seed=5)
    leaves = (x, w13, w2, w8, b8)

    def step():
        y = ops.feed_forward(x, w13, w2, None, None, None, "geglu", "paired", save)[0]
        z = ops.linear_fp8(y, w8, b8, x)[0]
        return (z.detach(), *torch.autograd.grad(z, leaves, d))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        n(300, 300) @ n(300, 300, seed=1)
        torch.cuda.synchronize()

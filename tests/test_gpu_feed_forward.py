"""The operators around the GLU as torch ops and together: the ops against the binding, opcheck, graph
capture, and the example's feed-forward blocks against plain FP32 torch."""
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


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_ops_equal_the_binding_and_carry_its_gradients(gpu):
    x, y, w, d = n(48, 264), n(48, 264, seed=1), n(264, seed=2), n(48, 264, seed=3)
    out = ops.block_norm(x, y, w, w, w, w, True, 0.5, "layer")
    want = gpu.glu_block_norm(x, y, gate=w, w_pre=w, b_pre=w, w_post=w, post=True, res_scale=0.5, kind="layer")
    assert same(out, want)
    leaves = [t.clone().requires_grad_(True) for t in (x, y, w, w, w, w)]
    xo, h, _ = ops.block_norm(*leaves, True, 0.5, "layer")
    got = torch.autograd.grad([xo, h], leaves, [d, d])
    dx, dy, dgate, dwp, dw, db = gpu.glu_block_norm_bwd(x, y, want[2], d, d, gate=w, w_pre=w, b_pre=w, w_post=w,
                                                        post=True, res_scale=0.5, kind="layer")
    assert same(got, (dx, dy, dgate, dw, db, dwp))
    a = x.clone().requires_grad_(True)
    _, h, st = ops.block_norm(a)
    assert same(torch.autograd.grad(h, a, d), gpu.glu_block_norm_bwd(x, None, st, None, d)[:1])

    wt, b, off = n(3, 72, 264, seed=4, scale=0.06), n(3, 72, seed=5), torch.tensor([0, 20, 20, 48], dtype=torch.int32).cuda()
    dy = n(48, 72, seed=6)
    leaves = [t.clone().requires_grad_(True) for t in (x, wt, b)]
    out, pre = ops.linear(*leaves, None, off, "gelu")
    want, wpre = gpu.glu_linear(x, wt, b, act="gelu", offsets=off, save_pre=True)
    assert same((out, pre), (want, wpre))
    assert same(torch.autograd.grad(out, leaves, dy),
                gpu.glu_linear_bwd(dy, x, wt, pre=wpre, act="gelu", offsets=off, bias=True))
    res = n(48, 72, seed=7).requires_grad_(True)
    out, _ = ops.linear(x, wt[0], None, res)
    assert same(torch.autograd.grad(out, res, dy), (dy,))
    with pytest.raises(RuntimeError):
        leaf = x.clone().requires_grad_(True)
        ops.linear(leaf, wt[0], None, None, None, "silu", False)[0].sum().backward()

    ids = torch.randint(-1, 5, (48, 3), device="cuda")
    rows, offsets = ops.moe_sort(ids, 5)
    assert same((rows, offsets), gpu.glu_moe_sort(ids, 5))
    a, wts = x.clone().requires_grad_(True), torch.rand(48, 3, device="cuda", requires_grad=True)
    xs = ops.moe_permute(a, rows, offsets)
    out = ops.moe_combine(xs, rows, offsets, wts, y)
    assert same((out,), (gpu.glu_moe_combine(xs.detach(), rows, wts.detach(), y),))
    da, dw = torch.autograd.grad(out, (a, wts), d)
    dys, dww = gpu.glu_moe_combine_bwd(d, xs.detach(), rows, wts.detach(), offsets)
    assert same((dw, da), (dww, gpu.glu_moe_combine(dys, rows)))
    ys = n(144, 264, seed=9).requires_grad_(True)
    assert same(torch.autograd.grad(ops.moe_combine(ys, rows, offsets), ys, d), (gpu.glu_moe_permute(d, rows, offsets),))


def test_opcheck(gpu):
    x, w = n(24, 72), n(72, seed=1)
    utils = ("test_schema", "test_faketensor", "test_autograd_registration")
    torch.library.opcheck(ops.block_norm.default, (x, x.clone(), w, w.clone(), None, w.clone(), True), test_utils=utils)
    torch.library.opcheck(ops.block_norm.default, (x,), test_utils=utils)
    torch.library.opcheck(ops.linear.default, (x, n(40, 72, seed=2), None, None, None, "silu"), test_utils=utils)
    ids = torch.randint(0, 4, (24, 2), device="cuda", dtype=torch.int32)
    torch.library.opcheck(ops.moe_sort.default, (ids, 4), test_utils=utils)
    rows, offsets = ops.moe_sort(ids, 4)
    torch.library.opcheck(ops.moe_permute.default, (x, rows, offsets), test_utils=utils)
    torch.library.opcheck(ops.moe_combine.default, (n(48, 72), rows, offsets, torch.rand(24, 2, device="cuda")),
                          test_utils=utils)


def plain_block(x, y, p, choices):
    """example.feed_forward in FP32 torch."""
    def rms(t):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6)

    xo = x + p["gate"] * rms(y) * p["w_post"]
    h = rms(xo) * p["w_pre"]

    def expert(t, w13, w2, b2):
        a = t @ w13.t()
        inner = w13.shape[0] // 2
        return (torch.nn.functional.silu(a[:, :inner]) * a[:, inner:]) @ w2.t() + b2

    if not choices:
        return xo, expert(h, p["w13"], p["w2"], p["b2"])
    top, ids = torch.topk(h @ p["router"].t(), choices, dim=1)
    weights = torch.softmax(top, dim=1)
    out = 0
    for e in range(p["router"].shape[0]):
        share = (weights * (ids == e)).sum(1, keepdim=True)
        out = out + share * expert(h, p["w13"][e], p["w2"][e], p["b2"][e])
    return xo, out


@pytest.mark.parametrize("experts,choices", [(0, 0), (6, 2)])
def test_block_against_plain_torch(gpu, experts, choices):
    """Output and every gradient of a block.  Five BF16 roundings lie between the inputs and the output and
    as many between the loss and a gradient: each moves a tensor by at most 2^-8 of itself, 2^-9.5
    on average, so 10 of them stay under 2^-6 in the 2-norm.  Experts are compared where both
    sides choose the same ones (a router logit may be rounded across a tie), and to 2^-4: their
    logits, up to 16 here, are rounded too, which moves a softmax weight by up to 2^-5 of itself."""
    p = example.make_params(200, 328, experts)
    x, y, d = n(150, 200, seed=1), n(150, 200, seed=2), n(150, 200, seed=3)
    f = {k: t.detach().float().requires_grad_(True) for k, t in p.items()}
    if experts:   # push the logits apart, so that rounding does not change a choice
        with torch.no_grad():
            p["router"] *= 8
            f["router"] *= 8
    a, b = (t.clone().requires_grad_(True) for t in (x, y))
    fa, fb = (t.float().requires_grad_(True) for t in (x, y))
    got, want = example.feed_forward(a, b, p, choices), plain_block(fa, fb, f, choices)
    names = [k for k in p if k != "router"]
    gg = torch.autograd.grad(got, [a, b] + [p[k] for k in names], [d, d])
    wg = torch.autograd.grad(want, [fa, fb] + [f[k] for k in names], [d.float(), d.float()])
    if experts:
        with torch.no_grad():
            h = ops.block_norm(x, y, p["gate"], p["w_pre"], None, p["w_post"], True)[1]
            mine = torch.topk((h @ p["router"].t()).float(), choices, dim=1)[1].sort(1)[0]
            xo = x.float() + f["gate"] * (y.float() * torch.rsqrt(y.float().square().mean(1, keepdim=True) + 1e-6))
            hf = xo * torch.rsqrt(xo.square().mean(1, keepdim=True) + 1e-6)
            theirs = torch.topk(hf @ f["router"].t(), choices, dim=1)[1].sort(1)[0]
        agree = (mine == theirs).all(1)
        assert agree.float().mean() > 0.9
        got, want = [t[agree] for t in got], [t[agree] for t in want]
        gg, wg = [gg[0][agree], gg[1][agree]], [wg[0][agree], wg[1][agree]]
    for u, v in zip(list(got) + list(gg), list(want) + list(wg)):
        assert (u.float() - v).norm() <= 2.0 ** -6 * v.norm() * (4 if experts else 1)


def test_example_learns(gpu):
    for kw in (dict(), dict(experts=8, choices=2)):
        losses = example.train(steps=6, **kw)
        assert losses[-1] < 0.9 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))


def test_norm_feeds_the_block_scaled_gemm(gpu):
    """block_norm_mxfp8's codes and scales are glu_gemm's X operand."""
    import synthetic_inputs as si
    x, y, w = n(130, 256), n(130, 256, seed=1), n(256, seed=2)
    wq, ws = si.mx_operand(2 * 128, 256, seed=3, device="cuda")
    _, q, s, _ = gpu.glu_block_norm_mxfp8(x, y, w_pre=w)
    _, h, _ = gpu.glu_block_norm(x, y, w_pre=w)
    q2, _, s2, _ = gpu.glu_quant_mxfp8_f32(h.float(), rowwise=True)
    assert torch.equal(gpu.glu_gemm(q, s, wq, ws), gpu.glu_gemm(q2, s2, wq, ws))


def test_graph_replays_equal_eager(gpu):
    """A block with experts captured whole, with torch's topk and softmax kept outside: replays with eager
    work and overwritten outputs in between equal the eager results."""
    T, H, inner, E, k = 96, 264, 200, 6, 2
    x, y, w = n(T, H), n(T, H, seed=1), n(H, seed=2)
    w13, w2 = n(E, 2 * inner, H, seed=3, scale=0.06), n(E, H, inner, seed=4, scale=0.07)
    one, two = n(40, 2056, seed=5), n(136, 2056, seed=6, scale=0.02)   # a sum split over workgroups
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    wts, d = torch.rand(T, k, device="cuda"), n(T, H, seed=7)

    def step():
        xo, h, st = gpu.glu_block_norm(x, y, w_pre=w, w_post=w, post=True)
        rows, off = gpu.glu_moe_sort(ids, E)
        xs = gpu.glu_moe_permute(h, rows, off)
        a, pre = gpu.glu_linear(xs, w13, act="silu", offsets=off, save_pre=True)
        z = gpu.glu_fwd(a[:, :inner], a[:, inner:])
        ys = gpu.glu_linear(z, w2, offsets=off)
        out = gpu.glu_moe_combine(ys, rows, wts, xo)
        dys, dw = gpu.glu_moe_combine_bwd(d, ys, rows, wts, off)
        dz, dw2, _ = gpu.glu_linear_bwd(dys, z, w2, offsets=off)
        da = torch.empty_like(a)
        gpu.glu_bwd(a[:, :inner], a[:, inner:], dz, out=(da[:, :inner], da[:, inner:]))
        dxs, dw13, db = gpu.glu_linear_bwd(da, xs, w13, pre=pre, act="silu", offsets=off, bias=True)
        dh = gpu.glu_moe_combine(dxs, rows)
        grads = gpu.glu_block_norm_bwd(x, y, st, d, dh, w_pre=w, w_post=w, post=True)
        long = gpu.glu_linear(one.repeat(5, 1), two)
        return [out, dw, dw2, dw13, db, long] + [g for g in grads if g.numel()]

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    torch.cuda.synchronize()
    for replay in range(4):
        for t in outs:
            t.fill_(7.0)
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(outs, eager), f"replay {replay}"

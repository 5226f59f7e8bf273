"""The feed-forward op forms the gradients that are wanted and no others: each subset equal to the whole
backward's, and no product for what is not asked for."""
import itertools

import pytest
import torch

import glu_activation_microscaling_amd.torch_ops as torch_ops

pytestmark = pytest.mark.gpu
ops = torch.ops.glu_mx
BF16 = torch.bfloat16


def n(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


@pytest.mark.parametrize("offsets", [None, [3, 20, 20, 70]], ids=["dense", "groups"])
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_every_subset(gpu, monkeypatch, offsets, save):
    lead = () if offsets is None else (3,)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    leaves = (n(75, 136), n(*lead, 144, 136, seed=1, scale=0.1), n(*lead, 136, 72, seed=2, scale=0.1), n(*lead, 144, seed=3),
              n(*lead, 136, seed=4))
    dy = n(75, 136, seed=5)
    formed = []
    for name in ("_linear_bwd", "_gated_bwd"):
        f = getattr(torch_ops, name)
        monkeypatch.setattr(torch_ops, name, lambda *a, f=f, **k: formed.append(f(*a, **k)) or formed[-1])

    def gradients(need):
        t = [v.clone().requires_grad_(w) for v, w in zip(leaves, need)]
        formed.clear()
        y = ops.feed_forward(*t, off, "swiglu", "split", save)[0]
        got = torch.autograd.grad(y, [v for v, w in zip(t, need) if w], dy)
        return dict(zip([i for i, w in enumerate(need) if w], got))

    whole = gradients((True,) * 5)
    for need in itertools.product((False, True), repeat=5):
        if not any(need):
            continue
        got = gradients(need)
        assert all(torch.equal(g, whole[i]) for i, g in got.items()), need
        # of the size of w13 and w2: the gradients that were asked for alone
        shapes = [tuple(t.shape) for call in formed for t in call]
        assert shapes.count(tuple(leaves[1].shape)) == need[1] and shapes.count(tuple(leaves[2].shape)) == need[2], need
        # [75, 136] is dx alone; [75, 72] is dh, and h formed again for w2's gradient
        assert shapes.count((75, 136)) == need[0] and shapes.count((75, 72)) == (need[0] or need[1] or need[3]) + need[2], need


def test_opcheck_with_frozen_weights(gpu):
    x, w13, w2 = n(24, 72).requires_grad_(True), n(80, 72, seed=1, scale=0.1), n(72, 40, seed=2, scale=0.1)
    torch.library.opcheck(ops.feed_forward, (x, w13, w2, None, None, None, "swiglu", "split", "mxfp8"))
    torch.library.opcheck(ops.feed_forward, (x.detach(), w13, w2.requires_grad_(True), None, None, None, "swiglu", "split", "bf16"))
    h, pre, extra = ops.gated_linear(x.detach(), w13)
    for need in itertools.product((False, True), repeat=3):
        torch.library.opcheck(ops.feed_forward_backward, (n(24, 72, seed=3), x.detach(), w13, w2.detach(), pre, extra, None, "swiglu",
                                                          "split", False, True, *need))

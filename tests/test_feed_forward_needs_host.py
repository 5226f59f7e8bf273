"""Shapes of the feed-forward op's gradients when only some are wanted (no GPU)."""
import itertools

import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import glu_activation_microscaling_amd.torch_ops  # noqa: F401

ops = torch.ops.glu_mx


def test_what_is_not_wanted_is_zero_sized():
    def b(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    with FakeTensorMode():
        x, w13, w2, pre, extra = b(40, 64), b(144, 64), b(56, 72), b(40, 144), b(40, 72, dtype=torch.uint8)
        for need in itertools.product((False, True), repeat=5):
            g = ops.feed_forward_backward(b(40, 56), x, w13, w2, pre, extra, None, "swiglu", "split", need[3], need[4], *need[:3])
            want = [(40, 64), (144, 64), (56, 72), (144,), (56,)]
            assert [tuple(t.shape) for t in g] == [s if w else (0,) for s, w in zip(want, need)]


def test_gradients_are_asked_for_one_by_one():
    """Autograd asks the backward op for what has a leaf, and for nothing else."""
    from torch.fx.experimental.proxy_tensor import make_fx

    def f(*leaves):
        t = [v.detach().requires_grad_(i in wanted) for i, v in enumerate(leaves)]
        return torch.autograd.grad(ops.feed_forward(*t)[0].sum(), [t[i] for i in wanted])

    m = dict(device="meta", dtype=torch.bfloat16)
    leaves = [torch.empty(s, **m) for s in ((8, 64), (48, 64), (32, 24), (48,), (32,))]
    for wanted in ((0,), (2,), (4,), (0, 3), (1, 2, 3, 4), (0, 1, 2, 3, 4)):
        gm = make_fx(f)(*leaves)
        node = next(t for t in gm.graph.nodes if "feed_forward_backward" in str(t.target))
        args = list(node.args) + [True] * (14 - len(node.args))
        assert [args[i] for i in (11, 12, 13, 9, 10)] == [i in wanted for i in range(5)]

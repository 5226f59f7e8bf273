"""The torch ops around the GLU under torch.compile(fullgraph=True) (aot_eager: no generated kernels) and
torch.library.opcheck, its dispatch through autograd included."""
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


@pytest.mark.parametrize("experts,choices", [(0, 0), (6, 2)])
def test_a_block_compiles_whole_and_equals_eager(gpu, experts, choices):
    p = example.make_params(200, 328, experts)
    x, y, d = (n(150, 200, seed=i).requires_grad_(i < 2) for i in range(3))
    leaves = [x, y] + list(p.values())

    def step(x, y, p):
        return example.feed_forward(x, y, p, choices)

    eager = step(x, y, p)
    compiled = torch.compile(step, fullgraph=True, backend="aot_eager")(x, y, p)
    for a, b in zip(eager, compiled):
        assert torch.equal(a, b)
    for a, b in zip(torch.autograd.grad(eager, leaves, [d, d]), torch.autograd.grad(compiled, leaves, [d, d])):
        assert torch.equal(a, b)


def test_a_grouped_product_with_residual_and_rows_of_no_group_compiles(gpu):
    x, w, res = (t.requires_grad_(True) for t in (n(50, 64), n(3, 72, 64, seed=1), n(50, 72, seed=2)))
    off, dy = torch.tensor([4, 10, 10, 40], dtype=torch.int32, device="cuda"), n(50, 72, seed=3)

    def step(x, w, res):
        return ops.linear(x, w, None, res, off, "silu")[0]

    eager, compiled = step(x, w, res), torch.compile(step, fullgraph=True, backend="aot_eager")(x, w, res)
    assert torch.equal(eager, compiled)
    for a, b in zip(torch.autograd.grad(eager, (x, w, res), dy), torch.autograd.grad(compiled, (x, w, res), dy)):
        assert torch.equal(a, b)


def test_opcheck(gpu):
    x, y, w = n(24, 72).requires_grad_(True), n(24, 72, seed=1), n(72, seed=2)
    torch.library.opcheck(ops.block_norm, (x, y, w, w.clone(), w.clone(), w.clone(), True, 0.5, "layer"))
    torch.library.opcheck(ops.block_norm, (x,))
    torch.library.opcheck(ops.linear, (x, n(40, 72, seed=3), n(40, seed=4), n(24, 40, seed=5), None, "silu"))
    off = torch.tensor([2, 10, 20], dtype=torch.int32, device="cuda")
    torch.library.opcheck(ops.linear, (x, n(2, 40, 72, seed=3), None, n(24, 40, seed=5), off, "none"))
    ids = torch.randint(0, 4, (24, 2), device="cuda", dtype=torch.int32)
    torch.library.opcheck(ops.moe_sort, (ids, 4))
    rows, offsets = ops.moe_sort(ids, 4)
    torch.library.opcheck(ops.moe_permute, (x, rows, offsets))
    torch.library.opcheck(ops.moe_combine, (n(48, 72).requires_grad_(True), rows, offsets,
                                            torch.rand(24, 2, device="cuda"), y))

"""The rules that pick a product's kernel: the shapes that tests name a kernel for take it, and the parts of a
gradient's sum do not depend on the other gradient (no GPU)."""
import itertools

import pytest

import test_gpu_fp8_scales as scales
import test_gpu_gated_overflow as overflow
import test_gpu_large_tiles as large
from product_plans import available, plans

pytestmark = pytest.mark.skipif(not available, reason="g++ not available")


def test_large_tiles():
    queries, want = [], []
    for ops, cases in ((("gated", "gated8"), large.GATED), (("fp8",), large.FP8)):
        for (M, N, K, kernel), op in itertools.product(cases, ops):
            queries.append((op, M, N, K, 0))
            want.append((kernel, 1))
    for ops, cases in ((("gated", "gated8"), large.GATED_GROUPS), (("fp8",), large.FP8_GROUPS)):
        for (counts, before, after, N, K, kernel), op in itertools.product(cases, ops):
            queries.append((op, before + sum(counts) + after, N, K, len(counts)))
            want.append((kernel, 1))
    assert plans(queries) == want


def test_extremes_reach_every_kernel():
    tiles = {"256x256", "256x128", "128x128"}
    taken = plans([("fp8", M, N, K, 0 if off is None else len(off) - 1) for M, N, K, off in scales.SHAPES])
    assert {k for k, _ in taken} == tiles | {"32x128", "few rows"} and any(p > 1 for _, p in taken)
    taken = plans([("gated", *s, 0) for s in overflow.SHAPES])
    assert {k for k, _ in taken} == tiles | {"few rows"} and any(p > 1 for _, p in taken)
    assert plans([("fp8", M, N, 1 << 22, 0) for M, N in ((1, 16), (20, 136), (300, 264))]) == [("few rows", 1), ("128x128", 128),
                                                                                          ("256x256", 64)]


def test_each_kernel_is_taken_somewhere():
    sizes = [(M, N, K, 0) for M, N, K in itertools.product((1, 40, 300, 3000, 16384), (136, 1000, 7168), (264, 2048, 16384))]
    sizes += [(M, N, K, 16) for M, N, K in itertools.product((100, 4000, 16384), (1000, 2048), (264, 2048))]
    for op in ("linear", "gated", "gated8", "fp8"):
        taken = {k for k, _ in plans([(op, *s) for s in sizes])}
        assert taken == {"256x256", "256x128", "128x128", "32x128"} | (set() if op == "gated8" else {"few rows"}), op


def test_a_gradients_parts_do_not_depend_on_the_other():
    extents = (8, 64, 256, 512, 1000, 1024, 2048, 3000, 4096)
    sizes = [(M, N, K, 0) for M, N, K in itertools.product(extents, repeat=3)]
    both, dx, dw = (plans([(op, *s) for s in sizes]) for op in ("both", "dx", "dw"))
    joint = [i for i, (kernel, _) in enumerate(both) if kernel is not None]
    assert len(joint) > 50 and all(dx[i][1] == 1 and dw[i][1] == 1 for i in joint)
    assert sum(p > 1 for _, p in dx) > 50


def test_measured_shapes_take_the_fastest():
    """Calls whose times at each tile size and count of parts stand beside the rules."""
    fastest = {
        ("linear", 1000, 1000, 1000, 0): ("128x128", 1), ("linear", 512, 2048, 2048, 0): ("128x128", 1),
        ("linear", 1021, 1000, 2056, 0): ("128x128", 2), ("linear", 968, 2048, 4096, 0): ("128x128", 2),
        ("linear", 968, 2048, 16384, 0): ("256x128", 4), ("linear", 2048, 4096, 4096, 0): ("256x128", 1),
        ("linear", 4096, 4096, 1024, 0): ("256x256", 1), ("linear", 6000, 4096, 2048, 0): ("256x256", 1),
        ("linear", 5000, 4096, 1024, 0): ("256x256", 1), ("dx", 2048, 512, 8192, 0): ("256x256", 1),
        ("dx", 2048, 512, 2048, 0): ("128x128", 1), ("dw", 4096, 4096, 2048, 8): ("256x256", 1),
        ("linear", 8192, 4096, 1024, 16): ("256x256", 1), ("gated", 8192, 2048, 1024, 16): ("256x256", 1),
        ("gated8", 968, 1024, 2048, 0): ("128x128", 1), ("gated8", 2048, 2048, 4096, 0): ("256x128", 1),
        ("fp8", 6000, 4096, 2048, 0): ("256x256", 1), ("fp8", 16, 2048, 2048, 0): ("128x128", 4),
        ("fp8", 1021, 1000, 2048, 0): ("128x128", 1), ("fp8", 2048, 4096, 4096, 0): ("256x128", 1)}
    assert dict(zip(fastest, plans(list(fastest)))) == fastest

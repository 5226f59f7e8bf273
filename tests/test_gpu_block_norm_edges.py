"""The norms around a block on the GPU at extents out of the ordinary."""
import pytest
import torch

from test_gpu_block_norm import draw

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_no_rows_with_parameters_for_each_row(gpu):
    """Parameters [M, H] and M = 0: no rows come out, their gradients are [0, H], and those of the
    parameters for all rows are zero."""
    x, y, dxo, dh, p = draw(0, 520)
    p["gate"] = p["w_pre"] = torch.empty(0, 520, device="cuda", dtype=BF16)
    x_out, h, stats = gpu.glu_block_norm(x, y, post=True, **p)
    assert x_out.shape == h.shape == (0, 520) and stats.shape == (0, 4)
    dx, dy, dgate, dw_post, dw_pre, db_pre = gpu.glu_block_norm_bwd(x, y, stats, dxo, dh, post=True, **p)
    assert dx.shape == dy.shape == dgate.shape == dw_pre.shape == (0, 520)
    assert (dw_post == 0).all() and dw_post.shape == (520,) and (db_pre == 0).all() and db_pre.shape == (520,)
    none = torch.empty(0, 64, device="cuda", dtype=BF16)
    assert [t.shape for t in gpu.glu_block_norm_mxfp8(none, none, gate=none)] == [(0, 64), (0, 64), (0, 2), (0, 4)]


def test_parameters_of_no_rows_for_some_rows_are_refused(gpu):
    x, y, _, _, p = draw(4, 520)
    for name in ("gate", "w_pre", "b_pre"):
        with pytest.raises(ValueError):
            gpu.glu_block_norm(x, y, post=True, **dict(p, **{name: torch.empty(0, 520, device="cuda", dtype=BF16)}))
    x, y, _, _, p = draw(0, 520)
    with pytest.raises(ValueError):   # two numbers of groups
        gpu.glu_block_norm(x, y, gate=torch.empty(0, 520, device="cuda", dtype=BF16),
                           w_pre=torch.empty(3, 520, device="cuda", dtype=BF16))

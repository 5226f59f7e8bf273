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


@pytest.mark.parametrize("H", [32, 2048, 9984])
def test_mxfp8_is_the_quantizer_of_h_at_the_ends_of_the_range(gpu, H):
    """NaN, infinities, zeros of both signs, subnormals and values near BF16's largest in h, put there by the
    shift and the weight of the norm: the codes and scales are the quantizer's to the byte."""
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(12, H, generator=g, device="cuda").to(BF16)
    w = torch.exp2(torch.randint(-130, 120, (12, H), generator=g, device="cuda").float()).to(BF16)
    b = torch.zeros(12, H, device="cuda", dtype=BF16)
    b[1, 3], b[2, 5], b[3, 7] = float("nan"), float("inf"), float("-inf")
    w[4], b[4] = 0, 0
    b[5], w[5] = -0.0, 0
    w[6] = 2.0 ** -130
    w[7], b[7, 1] = 1.0, 3.3e38
    w[8], b[8, 31] = 2.0 ** 126, -3.3e38
    w[9], b[9] = 0, torch.full((H,), 1e-40, device="cuda")
    x[10, 0] = float("nan")
    x[11, 1] = float("inf")
    _, h, _ = gpu.glu_block_norm(x, w_pre=w, b_pre=b)
    _, q, s, _ = gpu.glu_block_norm_mxfp8(x, w_pre=w, b_pre=b)
    q_row, _, s_row, _ = gpu.glu_quant_mxfp8_f32(h.float(), rowwise=True)
    assert torch.equal(q, q_row) and torch.equal(s, s_row)

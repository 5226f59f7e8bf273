"""The norms around a block on the GPU against 64-bit references (ffn_reference.py)."""
import pytest
import torch

import ffn_reference as ref
from ffn_reference import assert_close

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TERMS = 64   # roundings on the way from the inputs to a result of one row, sums over a row included


def draw(M, H, groups=1, stream=BF16, params=BF16, post=True, bias=True, seed=0, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, dtype=BF16, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    def rows(dtype, scale=1.0):
        return n(M, ld or H, dtype=dtype, scale=scale)[:, :H]

    G = (groups, H) if groups != 1 else (H,)
    x, y = rows(stream, 2.0), rows(BF16, 0.7)
    p = dict(gate=n(*G, dtype=params, scale=0.3, shift=0.5), w_pre=n(*G, dtype=params, scale=0.2, shift=1.0),
             b_pre=n(*G, dtype=params, scale=0.1) if bias else None,
             w_post=n(H, dtype=params, scale=0.2, shift=1.0) if post else None)
    return x, y, rows(stream, 0.1), rows(BF16, 0.1), p


def check(gpu, x, y, dxo, dh, p, **kw):
    M = x.shape[0]
    x_out, h, stats = gpu.glu_block_norm(x, y, **p, **kw)
    want, _ = ref.norm_forward(x, y, **p, **kw)
    if y is not None:
        assert_close("x_out", x_out, *want["x_out"], TERMS)
    else:
        assert x_out is x
    pre = kw.get("pre", True)
    if pre:
        assert_close("h", h, *want["h"], TERMS)
    else:
        assert h.numel() == 0
    got = gpu.glu_block_norm_bwd(x, y, stats, dxo, dh if pre else None, **p, **kw)
    got = dict(zip(("dx", "dy", "dgate", "dw_post", "dw_pre", "db_pre"), got))
    grads = ref.norm_backward(x, y, dxo, dh, **p, **kw)
    for name, t in got.items():
        if name not in grads:
            assert t.numel() == 0, name
            continue
        terms = TERMS if name in ("dx", "dy") else TERMS + M
        assert_close(name, t, *grads[name], terms)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 31, 64, 100, 511, 512, 513, 1000, 2048, 4100, 8192, 8193, 10248, 16384])
def test_widths(gpu, H):
    check(gpu, *draw(5, H, seed=H), post=True, res_scale=0.75)


@pytest.mark.parametrize("M", [1, 2, 3, 17, 64, 257, 1021])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows(gpu, M, kind):
    check(gpu, *draw(M, 768, seed=M), post=True, kind=kind)


@pytest.mark.parametrize("stream", [BF16, F32])
@pytest.mark.parametrize("params", [BF16, F32])
@pytest.mark.parametrize("H", [640, 645, 9000])
def test_types(gpu, stream, params, H):
    check(gpu, *draw(33, H, stream=stream, params=params), post=True, kind="layer", res_scale=1.25)


@pytest.mark.parametrize("M,groups", [(12, 2), (12, 12), (900, 3), (520, 520), (2100, 700), (5000, 5000), (4096, 1024)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_groups(gpu, M, groups, kind):
    check(gpu, *draw(M, 264, groups=groups), post=True, kind=kind)


def test_group_of_one_parameter_only(gpu):
    x, y, dxo, dh, p = draw(60, 520, groups=4)
    p["w_pre"], p["b_pre"] = p["w_pre"][0].contiguous(), None
    check(gpu, x, y, dxo, dh, p, post=True)
    x, y, dxo, dh, p = draw(2048, 72, groups=1024)
    p["gate"] = p["gate"][0].contiguous()
    check(gpu, x, y, dxo, dh, p, post=True)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
def test_parts_left_out(gpu, post, pre):
    x, y, dxo, dh, p = draw(19, 520)
    if not pre:
        p["w_pre"] = p["b_pre"] = None
    if not post:
        p["w_post"] = None
    check(gpu, x, y, dxo, dh, p, post=post, pre=pre)
    bare = dict(gate=None, w_pre=None, b_pre=None, w_post=None)
    check(gpu, x, y, dxo, dh, bare, post=post, pre=pre)
    if pre and not post:
        check(gpu, x, None, dxo, dh, dict(bare, w_pre=p["w_pre"], b_pre=p["b_pre"]))
        check(gpu, x, None, None, dh, dict(bare, w_pre=p["w_pre"], b_pre=p["b_pre"]), kind="layer")


@pytest.mark.parametrize("ld", [520, 528, 531])
def test_strides(gpu, ld):
    check(gpu, *draw(21, 520, ld=ld), post=True)


def test_large_mean_keeps_its_digits(gpu):
    """Rows whose mean is 2^6 times their spread: the variance is a sum of squared differences."""
    x, y, dxo, dh, p = draw(9, 1024, stream=F32)
    check(gpu, x + 64.0, y, dxo, dh, p, post=True, kind="layer")


def test_zero_rows_and_one_nan_row(gpu):
    x, y, dxo, dh, p = draw(8, 512, bias=False)
    x[3], y[3] = 0, 0                            # 0 / sqrt(eps)
    y[5, 7], x[6, 0] = float("nan"), float("inf")
    x_out, h, stats = gpu.glu_block_norm(x, y, post=True, **p)
    assert (h[3] == 0).all() and (x_out[3] == 0).all()
    assert torch.isnan(h[5].float()).all() and not torch.isfinite(h[6].float()).all()
    keep = [0, 1, 2, 4, 7]
    x2, h2, _ = gpu.glu_block_norm(x[keep].contiguous(), y[keep].contiguous(), post=True, **p)
    assert torch.equal(h[keep], h2) and torch.equal(x_out[keep], x2)
    dx = gpu.glu_block_norm_bwd(x, y, stats, dxo, dh, post=True, **p)[0]
    assert torch.isfinite(dx[keep].float()).all() and torch.isfinite(dx[3].float()).all()


def test_no_rows(gpu):
    x, y, dxo, dh, p = draw(0, 520)
    x_out, h, stats = gpu.glu_block_norm(x, y, post=True, **p)
    assert x_out.shape == h.shape == (0, 520)
    _, _, dgate, dw_post, dw_pre, db_pre = gpu.glu_block_norm_bwd(x, y, stats, dxo, dh, post=True, **p)
    for t in (dgate, dw_post, dw_pre, db_pre):
        assert t.shape == (520,) and (t == 0).all()


@pytest.mark.parametrize("M,H", [(1, 32), (7, 96), (130, 2048), (33, 8192), (9, 9984)])
def test_mxfp8_is_the_quantizer_of_h(gpu, M, H):
    x, y, _, _, p = draw(M, H)
    x[0, :32] = 0
    y[0, :32] = 0
    x_out, h, stats = gpu.glu_block_norm(x, y, **p, post=True)
    x_q, q, s, stats_q = gpu.glu_block_norm_mxfp8(x, y, **p, post=True)
    q_row, _, s_row, _ = gpu.glu_quant_mxfp8_f32(h.float(), rowwise=True)
    assert torch.equal(x_out, x_q) and torch.equal(stats, stats_q)
    assert torch.equal(q, q_row) and torch.equal(s, s_row)


def test_gradient_against_differences(gpu):
    """The kernel's gradients along random directions against central differences of the forward
    definition in 64 bits."""
    x, y, dxo, dh, p = draw(24, 328, stream=F32, params=F32)
    kw = dict(post=True, kind="layer", res_scale=0.9)
    _, _, stats = gpu.glu_block_norm(x, y, **p, **kw)
    grads = gpu.glu_block_norm_bwd(x, y, stats, dxo, dh, **p, **kw)
    at = dict(x=x, y=y, **p)

    def loss(v):
        out, _ = ref.norm_forward(**v, **kw)
        return (out["x_out"][0] * dxo.double()).sum() + (out["h"][0] * dh.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in zip(("x", "y", "gate", "w_post", "w_pre", "b_pre"), grads):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        # h^2 / 6 of the third derivative (order 1 per element moved) beside the rounding of each
        # gradient element
        e = 1e-4
        lo, hi = (loss({**{k: t.double() for k, t in at.items()}, name: at[name].double() + d * v}) for d in (-e, e))
        slope, dot = (hi - lo) / (2 * e), (grad.double() * v).sum()
        tol = ref.half_ulp(grad) * (grad.double() * v).abs().sum() + 1e-5 * (grad.double() * v).abs().sum() + 1e-6
        assert (slope - dot).abs() <= tol, (name, slope.item(), dot.item(), tol.item())


def test_same_bits_again_and_on_another_stream(gpu):
    x, y, dxo, dh, p = draw(700, 2056)

    def run():
        x_out, h, stats = gpu.glu_block_norm(x, y, **p, post=True)
        return (x_out, h) + gpu.glu_block_norm_bwd(x, y, stats, dxo, dh, **p, post=True)

    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    torch.cuda.current_stream().wait_stream(s)
    for t, u in zip(a, b):
        assert torch.equal(t, u)


def test_offsets_past_32_bits(gpu):
    """140000 rows of 16384: x, y and h are 4.6 GB each; the last rows are read and written in place."""
    M, H = 140000, 16384
    w = torch.ones(H, device="cuda", dtype=BF16)
    x = torch.empty(M, H, device="cuda", dtype=BF16)
    for i in range(0, M, 20000):
        x[i:i + 20000] = torch.randn(20000, H, device="cuda", dtype=BF16)
    x_out, h, stats = gpu.glu_block_norm(x, x, w_pre=w, gate=w)
    pick = [0, 65535, 65536, 131071, 131072, M - 1]
    x2, h2, _ = gpu.glu_block_norm(x[pick].contiguous(), x[pick].contiguous(), w_pre=w, gate=w)
    assert torch.equal(h[pick], h2) and torch.equal(x_out[pick], x2)
    del x_out
    dx = gpu.glu_block_norm_bwd(x, x, stats, h, h, w_pre=w, gate=w)[0]
    dx2 = gpu.glu_block_norm_bwd(x[pick].contiguous(), x[pick].contiguous(), stats[pick].contiguous(), h2, h2,
                                 w_pre=w, gate=w)[0]
    assert torch.equal(dx[pick], dx2)

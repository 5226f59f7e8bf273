"""8-bit checkpoints of the GLU's operands on the GPU: codes and scales against the oracle's MXFP8
quantizer, the backward against the definition in 64 bits and against the BF16 GLU at the
values that the codes stand for."""
import numpy as np
import pytest
import torch

import gated_reference as ref
import oracle
from ffn_reference import BF16_HALF_ULP, D

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def draw(M, N, seed=0, ld=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    big = torch.where(torch.rand(N, generator=g, device="cuda") < 0.03, 30.0, 1.0)

    def n(scale=1.0):
        return (torch.randn((M, N + ld), generator=g, device="cuda") * scale).to(BF16)[:, :N]
    return (n() * big).to(BF16) if not ld else n(3.0), n(), n(0.1)


def padded(t):
    """FP32, columns filled up to whole blocks of 32 with zeros."""
    return torch.nn.functional.pad(t.float(), (0, -t.shape[1] % 32)).cpu().numpy()


def check_codes(q, s, gate, up):
    M, N = gate.shape
    NB = (N + 31) // 32
    for h, t in enumerate((gate, up)):
        wq, ws = oracle.quant_mxfp8(padded(t), 1)[:2]
        assert np.array_equal(q[:, h * N:(h + 1) * N].cpu().numpy(), wq.reshape(M, -1)[:, :N]), ("codes", h)
        assert np.array_equal(s[:, h * NB:(h + 1) * NB].cpu().numpy(), ws.reshape(M, NB)), ("scales", h)


def paired(gate, up):
    return torch.stack([gate, up], 2).flatten(1).contiguous()


SHAPES = [(1, 8), (1, 32), (3, 40), (7, 64), (8, 264), (33, 1000), (64, 72), (130, 2048), (257, 4104), (1021, 1000)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("act", ref.ACTS)
def test_shapes(gpu, M, N, act):
    gate, up, dh = draw(M, N, seed=M + N)
    h, q, s = gpu.glu_fwd_ckpt(gate, up, act=act)
    assert torch.equal(h, gpu.glu_fwd(gate, up, act=act))
    check_codes(q, s, gate, up)
    d, again = gpu.glu_bwd_ckpt(q, s, dh, act=act, need_h=True)
    g, u = ref.restored(q, s, N)
    # the restored values are BF16 numbers: the BF16 GLU's own results, bit for bit
    da, db = gpu.glu_bwd(g.to(BF16), u.to(BF16), dh, act=act)
    assert torch.equal(g.to(BF16).to(D), g) and torch.equal(u.to(BF16).to(D), u)
    assert torch.equal(d, torch.cat([da, db], 1)) and torch.equal(again, gpu.glu_fwd(g.to(BF16), u.to(BF16), act=act))
    # and the formulas
    dd = dh.to(D)
    for got, want, off in ((d[:, :N], dd * u * ref.act_grad(g, act), (dd * u).abs()),
                           (d[:, N:], dd * ref.act(g, act), (dd * g).abs()),
                           (again, ref.act(g, act) * u, (g * u).abs())):
        tol = BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + ref.rounding(g, act) * off + 2.0 ** -120
        assert ((got.to(D) - want).abs() <= tol).all()


@pytest.mark.parametrize("M,N", [(1, 8), (5, 72), (130, 264)])
def test_layouts_strides_and_without_h(gpu, M, N):
    gate, up, dh = draw(M, N, seed=1, ld=16)
    h, q, s = gpu.glu_fwd_ckpt(gate, up)
    check_codes(q, s, gate, up)
    hp, qp, sp = gpu.glu_fwd_ckpt(paired(gate, up), layout="paired")
    assert torch.equal(h, hp) and torch.equal(q, qp) and torch.equal(s, sp)
    none, q2, s2 = gpu.glu_fwd_ckpt(gate, up, need_h=False)
    assert none.numel() == 0 and torch.equal(q, q2) and torch.equal(s, s2)
    out = torch.full((M, N + 8), 7.0, dtype=BF16, device="cuda")
    gpu.glu_fwd_ckpt(gate, up, out=out[:, :N])
    assert torch.equal(out[:, :N], h) and (out[:, N:] == 7.0).all()
    d, none = gpu.glu_bwd_ckpt(q, s, dh)
    dp, _ = gpu.glu_bwd_ckpt(q, s, dh, layout="paired")
    assert none.numel() == 0 and torch.equal(dp, paired(d[:, :N].contiguous(), d[:, N:].contiguous()))
    big = torch.full((M, 2 * N + 24), 7.0, dtype=BF16, device="cuda")
    gpu.glu_bwd_ckpt(q, s, dh, out=big[:, :2 * N])
    assert torch.equal(big[:, :2 * N], d) and (big[:, 2 * N:] == 7.0).all()


def test_extreme_and_non_finite_blocks(gpu):
    gate, up, dh = draw(6, 200, seed=3)
    gate[0, 5], gate[1, 190], up[2, 32], up[3, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    gate[4] = 0.0
    up[4] *= 2.0 ** -130
    gate[5] *= 2.0 ** 100
    up[5] *= 2.0 ** -110
    _, q, s = gpu.glu_fwd_ckpt(gate, up)
    check_codes(q, s, gate, up)
    g, u = ref.restored(q, s, 200)
    assert torch.isnan(g[0, :32]).all() and not torch.isnan(g[0, 32:]).any()
    assert torch.isnan(g[1, 192 - 32:192]).all() and not torch.isnan(g[1, 192:]).any()
    d, again = gpu.glu_bwd_ckpt(q, s, dh, need_h=True)
    da, db = gpu.glu_bwd(g.to(BF16), u.to(BF16), dh)
    for got, want in ((d[:, :200], da), (d[:, 200:], db), (again, gpu.glu_fwd(g.to(BF16), u.to(BF16)))):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


def test_no_rows(gpu):
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    h, q, s = gpu.glu_fwd_ckpt(e, e)
    assert h.shape == (0, 64) and q.shape == (0, 128) and s.shape == (0, 4)
    d, again = gpu.glu_bwd_ckpt(q, s, e, need_h=True)
    assert d.shape == (0, 128) and again.shape == (0, 64)

"""Quantizers to E4M3 with a scale for each 128, bit for bit against the definition, and products of
such operands against 64-bit sums (fp8_reference.py)."""
import pytest
import torch

import fp8_reference as ref
from ffn_reference import BF16_HALF_ULP, D, segments

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(M, N, seed=0, ld=0):
    g = gen(seed)
    t = torch.randn((M, N + ld), generator=g, device="cuda")
    t = t * torch.where(torch.rand(N + ld, generator=g, device="cuda") < 0.01, 25.0, 1.0)
    return t.to(BF16)[:, :N]


def check_quant(got, x, rowwise, colwise):
    M, N = x.shape
    q_row, q_col, s_row, s_col = got
    if rowwise:
        q, s = ref.quant(x, 1, 128)
        assert torch.equal(q_row[:, :N], q) and (q_row[:, N:] == 0).all()
        assert torch.equal(s_row.view(torch.int32), s.t().contiguous().view(torch.int32))
    else:
        assert q_row.numel() == 0 and s_row.numel() == 0
    if colwise:
        q, s = ref.quant(x, 128, 1)
        assert torch.equal(q_col[:, :M], q.t()) and (q_col[:, M:] == 0).all()
        assert torch.equal(s_col.view(torch.int32), s.view(torch.int32))
    else:
        assert q_col.numel() == 0 and s_col.numel() == 0


MODES = [(True, False), (False, True), (True, True)]
SHAPES = [(1, 8), (1, 128), (7, 120), (16, 136), (64, 1000), (127, 256), (129, 264), (300, 2056), (1021, 1000)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("rowwise,colwise", MODES)
def test_quant(gpu, M, N, rowwise, colwise):
    x = matrix(M, N, seed=M + N)
    got = gpu.glu_quant_fp8(x, rowwise=rowwise, colwise=colwise)
    assert got[0].numel() == 0 or got[0].shape == (M, (N + 15) // 16 * 16)
    check_quant(got, x, rowwise, colwise)


def test_every_quotient_of_two_bf16_numbers(gpu):
    """Each significand against each largest one, over the exponents down to E4M3's subnormals: every tie
    there is, and every nearest miss of one."""
    sig = torch.arange(128, 256, dtype=torch.float32, device="cuda") / 128.0
    exps = torch.arange(-19, 1, device="cuda")
    top = sig.repeat_interleave(20)                                   # the row's largest magnitude
    x = (sig[None, :] * torch.exp2(exps.float()).repeat(128)[:, None]).expand(128 * 20, 128).clone()
    x = torch.where(x > top[:, None], x / 2, x)
    x[:, 0] = top
    x[:, 1::2] *= -1
    x = x.to(BF16)
    check_quant(gpu.glu_quant_fp8(x), x, True, False)
    y = x.t().contiguous()
    check_quant(gpu.glu_quant_fp8(y, rowwise=False, colwise=True), y, False, True)


@pytest.mark.parametrize("rowwise,colwise", MODES)
def test_quant_of_extremes(gpu, rowwise, colwise):
    x = matrix(300, 400, seed=5)
    x[:128, :128] = 0.0
    x[128:256, :128] *= 2.0 ** -126
    x[:128, 128:256] *= 2.0 ** 120
    x[130, 200], x[257, 300], x[3, 399] = float("nan"), float("inf"), -float("inf")
    x[256:, 256:384] *= 2.0 ** -101
    check_quant(gpu.glu_quant_fp8(x, rowwise=rowwise, colwise=colwise), x, rowwise, colwise)


@pytest.mark.parametrize("M,N", [(3, 72), (130, 264), (257, 1000)])
@pytest.mark.parametrize("act", ["swiglu", "geglu", "geglu_erf", "relu2"])
def test_glu(gpu, M, N, act):
    gate, up = matrix(M, N, seed=1, ld=16), matrix(M, N, seed=2, ld=16)
    h = gpu.glu_fwd(gate, up, act=act)
    pair = torch.stack([gate, up], 2).flatten(1).contiguous()
    for rowwise, colwise in MODES:
        got = gpu.glu_fwd_fp8(gate, up, act=act, rowwise=rowwise, colwise=colwise)
        check_quant(got, h, rowwise, colwise)
        for a, b in zip(got, gpu.glu_fwd_fp8(pair, act=act, layout="paired", rowwise=rowwise, colwise=colwise)):
            assert torch.equal(a, b)


def test_strides_and_no_rows(gpu):
    x = matrix(70, 136, seed=3, ld=24)
    check_quant(gpu.glu_quant_fp8(x, colwise=True), x, True, True)
    e = x[:0]
    got = gpu.glu_quant_fp8(e, colwise=True)
    assert [tuple(t.shape) for t in got] == [(0, 144), (136, 0), (2, 0), (0, 136)]


@pytest.mark.parametrize("N,K", [(8, 8), (120, 136), (128, 128), (264, 1000), (1000, 264)])
@pytest.mark.parametrize("groups", [None, 3])
def test_weights(gpu, N, K, groups):
    w = matrix((groups or 1) * N, K, seed=N).contiguous()
    w[0, 0] *= 2.0 ** 20
    if groups:
        w = w.reshape(groups, N, K)
        w[1, N - 1, K - 1] = float("nan")
    q, s, qt, st = gpu.glu_quant_fp8_weight(w, transpose=True)
    q2, s2, none, _ = gpu.glu_quant_fp8_weight(w)
    assert torch.equal(q, q2) and torch.equal(s.view(torch.int32), s2.view(torch.int32)) and none.numel() == 0
    for e in range(groups or 1):
        at = (lambda t: t[e]) if groups else (lambda t: t)
        wq, ws = ref.quant(at(w), 128, 128)
        assert torch.equal(at(q)[:, :K], wq) and (at(q)[:, K:] == 0).all()
        assert torch.equal(at(qt)[:, :N], wq.t()) and (at(qt)[:, N:] == 0).all()
        assert torch.equal(at(s).view(torch.int32), ws.view(torch.int32))
        assert torch.equal(at(st).view(torch.int32), ws.t().contiguous().view(torch.int32))


# ---- products --------------------------------------------------------------------------------

def operands(M, N, K, w_scales="block", groups=None, seed=0):
    """Codes and scales of every size of values, and bias and residual."""
    g = gen(seed)
    lead = () if groups is None else (groups,)
    kb = (K + 127) // 128

    def codes(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(ref.E4M3).view(torch.uint8)

    def scales(*shape):
        return torch.exp(torch.randn(shape, generator=g, device="cuda")) * 2.0 ** -8

    ws = scales(*lead, (N + 127) // 128, kb) if w_scales == "block" else scales(*lead, kb, N)
    return dict(xq=codes(M, K), xs=scales(kb, M), wq=codes(*lead, N, K), ws=ws,
                bias=(torch.randn((*lead, N), generator=g, device="cuda") * 10).to(BF16),
                residual=(torch.randn((M, N + 8), generator=g, device="cuda") * 10).to(BF16)[:, :N])


def check_product(gpu, t, w_scales="block", offsets=None, bias=True, residual=True):
    b, r = t["bias"] if bias else None, t["residual"] if residual else None
    y = gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"], b, r, w_scales=w_scales, offsets=offsets)
    M, N = y.shape
    want, err = torch.zeros(M, N, dtype=D, device="cuda"), torch.zeros(M, N, dtype=D, device="cuda")
    for e, i, j in segments(M, offsets):
        w, s, be = (t["wq"], t["ws"], b) if offsets is None else (t["wq"][e], t["ws"][e], None if b is None else b[e])
        v, x, terms = ref.product(t["xq"][i:j], t["xs"][:, i:j], w, s, w_scales)
        if be is not None:
            v, x = v + be.to(D), x + 2.0 ** -22 * (terms + be.to(D).abs())
        if r is not None:
            v, x = v + r[i:j].to(D), x + 2.0 ** -22 * (terms + r[i:j].to(D).abs())
        want[i:j], err[i:j] = v, x
    off = (y.to(D) - want).abs()
    tol = BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err
    assert not (off > tol).any(), (int((off > tol).sum()), (off > tol).nonzero()[0].tolist())
    return y


# few rows, each tile size and their edges; sums split, ragged and shorter than a block
PRODUCTS = [(1, 8, 16), (1, 24, 128), (2, 16, 144), (5, 1000, 4096), (8, 520, 1040), (8, 136, 2064), (9, 40, 128), (17, 136, 1040),
            (33, 512, 64), (64, 248, 2048), (65, 64, 4112), (100, 1000, 208), (128, 128, 144), (300, 520, 1104), (511, 72, 4112),
            (777, 1032, 528), (2500, 1032, 336), (3000, 4096, 64), (4000, 2008, 528), (300, 264, 16384)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("w_scales", ["block", "row"])
def test_products(gpu, M, N, K, w_scales):
    check_product(gpu, operands(M, N, K, w_scales, seed=M + K), w_scales)


@pytest.mark.parametrize("M", [1, 3, 8, 31, 200])
def test_epilogue(gpu, M):
    t = operands(M, 264, 400, seed=M)
    check_product(gpu, t, bias=False)
    check_product(gpu, t, residual=False)
    y = check_product(gpu, t, bias=False, residual=False)
    out = torch.full((M, 272), 7.0, dtype=BF16, device="cuda")
    gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"], out=out[:, :264])
    assert torch.equal(out[:, :264], y) and (out[:, 264:] == 7.0).all()


def offsets_of(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


GROUPS = [([40, 50, 60], 0), ([0, 130, 0, 0, 257, 1, 0], 0), ([300, 0], 0), ([1] * 70, 0), ([2, 0, 1] * 43, 7), ([100, 200], 150),
          ([0, 0, 0], 40), ([0], 0), ([1500, 1, 1300, 900], 0)]


@pytest.mark.parametrize("counts,after", GROUPS, ids=[str(i) for i in range(len(GROUPS))])
@pytest.mark.parametrize("N,K,w_scales", [(136, 208, "block"), (72, 1040, "row"), (384, 1024, "block")])
def test_groups(gpu, counts, after, N, K, w_scales):
    M = sum(counts) + after
    t = operands(M, N, K, w_scales, len(counts), seed=M)
    off = offsets_of(counts)
    y = check_product(gpu, t, w_scales, off)
    if after:                                    # rows of no group: whatever they hold, zeros come out
        assert (y[M - after:] == 0).all()
        t["xq"][M - after:], t["xs"][:, M - after:] = 0x7f, float("nan")
        again = gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"], t["bias"], t["residual"], w_scales=w_scales, offsets=off)
        assert torch.equal(y, again)


def test_lengths_of_zero(gpu):
    t = operands(0, 64, 80)
    assert gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"]).shape == (0, 64)
    for M in (5, 200):
        check_product(gpu, operands(M, 64, 0))   # a sum of no terms: bias and residual alone
        t = operands(M, 0, 64)
        assert gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"]).shape == (M, 0)


@pytest.mark.parametrize("M", [3, 150])
def test_nan_stays_in_its_row(gpu, M):
    t = operands(M, 136, 528)
    y = gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"])
    t["xs"][2, 1] = float("nan")
    z = gpu.glu_linear_fp8(t["xq"], t["xs"], t["wq"], t["ws"])
    assert torch.isnan(z[1]).all()
    keep = torch.arange(M, device="cuda") != 1
    assert torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("M,N,K", [(40, 72, 136), (260, 264, 520), (129, 1000, 264)])
def test_a_training_step(gpu, M, N, K):
    """y, dx and dW of one linear layer, each product on operands quantized along its sum."""
    x, w, dy = matrix(M, K, seed=1), (matrix(N, K, seed=2) * K ** -0.5).to(BF16).contiguous(), matrix(M, N, seed=3)
    xr, xc, sxr, sxc = gpu.glu_quant_fp8(x, colwise=True)
    wq, ws, wt, wts = gpu.glu_quant_fp8_weight(w, transpose=True)
    dr, dc, sdr, sdc = gpu.glu_quant_fp8(dy, colwise=True)

    def blocks(t, rows, cols):
        q, s = ref.quant(t, rows, cols)
        return ref.values(q) * s.to(D).repeat_interleave(rows, 0)[:t.shape[0]].repeat_interleave(cols, 1)[:, :t.shape[1]]

    W = blocks(w, 128, 128)
    for got, want, args in (
            (gpu.glu_linear_fp8(xr, sxr, wq, ws), blocks(x, 1, 128) @ W.t(), (xr, sxr, wq, ws, "block")),
            (gpu.glu_linear_fp8(dr, sdr, wt, wts), blocks(dy, 1, 128) @ W, (dr, sdr, wt, wts, "block")),
            (gpu.glu_linear_fp8(dc, sdc, xc, sxc, w_scales="row"), blocks(dy, 128, 1).t() @ blocks(x, 128, 1),
             (dc, sdc, xc, sxc, "row"))):
        v, err, _ = ref.product(*args)
        assert torch.allclose(v, want, rtol=1e-9, atol=1e-9 * float(want.abs().max()))
        assert ((got.to(D) - want).abs() <= BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err).all()

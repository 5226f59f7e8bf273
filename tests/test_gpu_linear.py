"""Linear products with their epilogue and gradients on the GPU against 64-bit references
(ffn_reference.py).  Products of BF16 values are exact in FP32, so a sum of K of them is within
K 2^-23 of the sum of their magnitudes whatever the order of the additions."""
import pytest
import torch

import ffn_reference as ref
from ffn_reference import assert_close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def draw(M, N, K, groups=None, seed=0, ld=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)

    lead = () if groups is None else (groups,)
    return dict(x=n(M, K + ld)[:, :K], w=n(*lead, N, K, scale=max(K, 1) ** -0.5), bias=n(*lead, N, scale=0.5),
                residual=n(M, N + ld)[:, :N], dy=n(M, N + ld, scale=0.1)[:, :N])


def offsets_of(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check_forward(gpu, t, act="none", offsets=None, bias=True, residual=True, save_pre=False):
    M, K = t["x"].shape
    b, r = t["bias"] if bias else None, t["residual"] if residual else None
    y = gpu.glu_linear(t["x"], t["w"], b, r, act=act, offsets=offsets, save_pre=save_pre)
    want, wpre = ref.linear_forward(t["x"], t["w"], b, r, act, offsets)
    if save_pre:
        y, pre = y
        assert pre.dtype == torch.float16
        assert_close("pre", pre, wpre[0], wpre[1], K + 2, 2.0 ** -25)   # FP16's subnormals
    assert_close("y", y, want[0], want[1], K + 8, want[2])
    return pre if save_pre else None


def check_backward(gpu, t, pre, act="none", offsets=None):
    M, N = t["dy"].shape
    K = t["x"].shape[1]
    got = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], pre=pre, act=act, offsets=offsets, bias=True)
    want = ref.linear_backward(t["dy"], t["x"], t["w"], pre, act, offsets)
    for name, a, terms in zip(("dx", "dw", "db"), got, (N, M, M)):
        v, s, e = want[name]
        assert_close(name, a, v, s, terms + 8, e)


# one row, few rows, each tile size and their edges; sums split, ragged and shorter than a step
SHAPES = [(1, 8, 8), (1, 24, 16), (2, 16, 72), (16, 40, 128), (17, 136, 1032), (33, 512, 64), (64, 248, 2048),
          (65, 128, 64), (100, 1000, 200), (128, 128, 136), (129, 264, 72), (300, 520, 1096), (511, 72, 4104),
          (777, 1032, 520), (2500, 2056, 328), (3000, 4096, 64), (4100, 2304, 136), (4000, 2056, 520),
          (4000, 4008, 4040)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(gpu, M, N, K):
    t = draw(M, N, K, seed=M + N)
    check_forward(gpu, t)
    check_backward(gpu, t, None)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_erf"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 264), (20, 520, 2056), (200, 264, 512), (200, 264, 1032), (2300, 2304, 264),
                                   (4000, 4008, 904)])
def test_activations(gpu, act, M, N, K):
    t = draw(M, N, K, seed=N)
    pre = check_forward(gpu, t, act, save_pre=act != "none")
    check_backward(gpu, t, pre, act)
    check_forward(gpu, t, act, bias=False, residual=False)
    check_forward(gpu, t, act, residual=False)


# groups: none empty; empty first, last and in between; one with all rows; many; few rows each;
# rows after the last group
GROUPS = [([40, 50, 60], 0), ([0, 130, 0, 0, 257, 1, 0], 0), ([0, 0, 300], 0), ([300, 0], 0), ([5, 0, 17, 64, 65, 3], 0),
          ([1] * 70, 0), ([2, 0, 1] * 43, 7), ([100, 200], 150), ([0, 0, 0], 40), ([0], 0), ([513, 255], 1),
          ([3000, 1, 2500, 900], 0)]


@pytest.mark.parametrize("counts,after", GROUPS, ids=[str(i) for i in range(len(GROUPS))])
@pytest.mark.parametrize("N,K", [(136, 200), (264, 64), (384, 1024), (72, 1032)])
def test_groups(gpu, counts, after, N, K):
    M = sum(counts) + after
    t = draw(M, N, K, groups=len(counts), seed=M)
    t["residual"] = t["residual"].contiguous()
    off = offsets_of(counts)
    if after:                                    # rows of no group: whatever they hold, zeros come out
        t["x"][M - after:] = float("nan")
        t["dy"][M - after:] = float("inf")
    for act in ("none", "silu"):
        pre = check_forward(gpu, t, act, off, save_pre=act != "none")
        check_backward(gpu, t, pre, act, off)


@pytest.mark.parametrize("M", [1, 7, 8, 9, 16, 31, 130])
@pytest.mark.parametrize("N,K", [(8, 4096), (520, 2048), (2056, 136), (4104, 1032)])
def test_few_rows(gpu, M, N, K):
    t = draw(M, N, K, seed=M, ld=8)
    pre = check_forward(gpu, t, "gelu", save_pre=True)
    check_backward(gpu, t, pre, "gelu")
    check_forward(gpu, t, "none", bias=False)


def test_groups_of_many_rows(gpu):
    counts = [2501, 3000, 0, 2099]
    t = draw(sum(counts), 2000, 2008, groups=4, seed=4)
    pre = check_forward(gpu, t, "silu", offsets_of(counts), save_pre=True)
    check_backward(gpu, t, pre, "silu", offsets_of(counts))


def test_offsets_out_of_range_are_clamped(gpu):
    t = draw(50, 64, 72, groups=3)
    off = torch.tensor([-5, 20, 1000, 2000], dtype=torch.int32, device="cuda")
    same = torch.tensor([0, 20, 50, 50], dtype=torch.int32, device="cuda")
    assert torch.equal(gpu.glu_linear(t["x"], t["w"], offsets=off), gpu.glu_linear(t["x"], t["w"], offsets=same))
    for a, b in zip(gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], offsets=off, bias=True),
                    gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], offsets=same, bias=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(3, 72, 136), (150, 136, 264), (2100, 2304, 72), (4000, 4008, 904)])
def test_strides(gpu, M, N, K):
    t = draw(M, N, K, ld=24)
    check_forward(gpu, t)
    check_backward(gpu, t, None)


def test_lengths_of_zero(gpu):
    t = draw(0, 64, 72)
    assert gpu.glu_linear(t["x"], t["w"], t["bias"]).shape == (0, 64)
    dx, dw, db = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], bias=True)
    assert dx.shape == (0, 72) and (dw == 0).all() and (db == 0).all()
    for M in (5, 200):                           # a sum of no terms: bias and residual alone
        t = draw(M, 64, 0)
        check_forward(gpu, t)
        dx, dw, db = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], bias=True)
        assert dx.shape == (M, 0) and dw.shape == (64, 0)
        t = draw(M, 0, 64)
        assert gpu.glu_linear(t["x"], t["w"]).shape == (M, 0)
        dx, dw, db = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], bias=True)
        assert (dx == 0).all() and dw.shape == (0, 64) and db.shape == (0,)


def test_gradients_one_by_one(gpu):
    t = draw(200, 136, 264)
    dx, dw, db = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], bias=True)
    a, b, c = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], need_dw=False)
    assert torch.equal(a, dx) and b.numel() == 0 and c.numel() == 0
    a, b, c = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], need_dx=False)
    assert a.numel() == 0 and torch.equal(b, dw) and c.numel() == 0
    a, b, c = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], need_dx=False, need_dw=False, bias=True)
    assert a.numel() == 0 and b.numel() == 0 and torch.equal(c, db)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_erf"])
def test_activation_at_its_ends(gpu, act):
    """Pre-activations from -1e30 to 1e30: act(p) for large |p| is p or 0, its gradient 1 or 0, and the
    saved pre-activation is clamped, not infinite."""
    v = torch.tensor([0.0, -0.0, 1e-30, 1e-6, 0.01, 1.0, 3.0, 9.0, 13.0, 20.0, 100.0, 3e4, 7e4, 1e10, 1e30],
                     device="cuda")
    p = torch.cat([v, -v])
    x = torch.zeros(p.numel(), 8, device="cuda", dtype=BF16)
    x[:, 0] = p.to(BF16)
    w = torch.zeros(8, 8, device="cuda", dtype=BF16)
    w[:, 0] = 1.0
    y, pre = gpu.glu_linear(x, w, act=act, save_pre=True)
    z = x[:, :1].double().expand(-1, 8)
    assert torch.equal(pre.double(), z.clamp(-65504, 65504).to(torch.float16).double())
    want = torch.where(z < -1000, torch.zeros_like(z), ref.act(z.clamp(min=-1000), act))
    assert ((y.double() - want).abs() <= ref.half_ulp(y) * want.abs() * 1.02 + ref.ACT_ERROR * z.abs().clamp(max=20)).all()
    dy = torch.ones(p.numel(), 8, device="cuda", dtype=BF16)
    _, _, db = gpu.glu_linear_bwd(dy, x, w, pre=pre, act=act, need_dx=False, need_dw=False, bias=True)
    grad = ref.act_grad(pre.double().clamp(-1000, 1000), act).sum(0)
    assert torch.isfinite(db.float()).all()
    assert ((db.double() - grad).abs() <= ref.half_ulp(db) * grad.abs() * 1.02 + ref.ACT_ERROR * p.numel()).all()


@pytest.mark.parametrize("M", [3, 150])
def test_nan_stays_in_its_row(gpu, M):
    t = draw(M, 136, 200)
    y = gpu.glu_linear(t["x"], t["w"], t["bias"], t["residual"], act="silu")
    t["x"][1, 5] = float("nan")
    z = gpu.glu_linear(t["x"], t["w"], t["bias"], t["residual"], act="silu")
    assert torch.isnan(z[1].float()).all()
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(y[keep], z[keep])


def test_gradient_against_differences(gpu):
    """The kernel's gradients along random directions against central differences in 64 bits."""
    t = draw(40, 136, 72)
    y, pre = gpu.glu_linear(t["x"], t["w"], t["bias"], act="gelu", save_pre=True)
    grads = gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], pre=pre, act="gelu", bias=True)
    at = {n: t[n].double() for n in ("x", "w", "bias")}

    def loss(v):
        return (ref.act(v["x"] @ v["w"].t() + v["bias"], "gelu") * t["dy"].double()).sum()

    g = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in zip(("x", "w", "bias"), grads):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        lo, hi = (loss({**at, name: at[name] + d * v}) for d in (-e, e))
        slope, dot = (hi - lo) / (2 * e), (grad.double() * v).sum()
        # each element is off by its own rounding, dp's and the saved pre-activation's
        tol = 3 * ref.BF16_HALF_ULP * (grad.double() * v).abs().sum()
        assert (slope - dot).abs() <= tol, (name, slope.item(), dot.item(), tol.item())


@pytest.mark.parametrize("M,N,K,groups", [(1, 2048, 4096, None), (300, 264, 1032, None), (2300, 2304, 264, None),
                                          (260, 136, 264, 5)])
def test_same_bits_again_and_on_another_stream(gpu, M, N, K, groups):
    t = draw(M, N, K, groups=groups)
    off = None if groups is None else offsets_of([M // groups] * groups)

    def run():
        y, pre = gpu.glu_linear(t["x"], t["w"], t["bias"], act="silu", offsets=off, save_pre=True)
        return (y, pre) + gpu.glu_linear_bwd(t["dy"], t["x"], t["w"], pre=pre, act="silu", offsets=off, bias=True)

    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_offsets_past_32_bits(gpu):
    """1.2 million rows of 2048 (4.9 GB): the first and last rows go through the same tiles as alone; the
    gradient of w sums over all of them."""
    M, N, K = 1200000, 64, 2048
    w = (torch.randn(N, K, device="cuda") * K ** -0.5).to(BF16)
    x = torch.zeros(M, K, device="cuda", dtype=BF16)
    dy = torch.zeros(M, N, device="cuda", dtype=BF16)
    last = 256
    x[-last:] = torch.randn(last, K, device="cuda").to(BF16)
    dy[-last:] = torch.randn(last, N, device="cuda").to(BF16)
    y = gpu.glu_linear(x, w)
    assert (y[:-last] == 0).all()
    want, _ = ref.linear_forward(x[-last:], w)
    assert_close("y", y[-last:], want[0], want[1], K)
    dx, dw, db = gpu.glu_linear_bwd(dy, x, w, bias=True)
    assert (dx[:-last] == 0).all()
    grads = ref.linear_backward(dy[-last:], x[-last:], w, None)
    for name, a, terms in (("dx", dx[-last:], N), ("dw", dw, M), ("db", db, M)):
        assert_close(name, a, *grads[name][:2], min(terms, 4096))

"""Gated projections and their gradients on the GPU against 64-bit references (gated_reference.py):
products of BF16 values are exact in FP32, so a sum of K of them is within K 2^-23 of the sum of
their magnitudes whatever the order, and that moves h by no more than the slopes of act(g) u."""
import pytest
import torch

import gated_reference as ref
from ffn_reference import BF16_HALF_ULP, D, assert_close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def draw(M, N, K, groups=None, seed=0, ld=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)

    lead = () if groups is None else (groups,)
    return dict(x=n(M, K + ld)[:, :K], w=n(*lead, 2 * N, K, scale=max(K, 1) ** -0.5), bias=n(*lead, 2 * N, scale=0.5),
                dh=n(M, N + ld, scale=0.1)[:, :N])


def offsets_of(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def close(name, got, want, err):
    tol = BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err + 2.0 ** -120
    bad = (got.to(D) - want).abs() > tol
    assert torch.isfinite(got.float()).all(), f"{name}: not finite"
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def check(gpu, t, act="swiglu", layout="split", save="bf16", offsets=None, bias=True):
    """Forward and backward of one call; returns their outputs."""
    M, K, N = *t["x"].shape, t["w"].shape[-2] // 2
    b = t["bias"] if bias else None
    p = dict(act=act, w_layout=layout, offsets=offsets)
    plain = gpu.glu_gated_linear(t["x"], t["w"], b, **p)
    (g, eg), (u, eu), (h, eh) = ref.forward(t["x"], t["w"], b, act, layout, offsets)
    close("h", plain, h, eh)
    if save == "none":
        return plain
    h2, pre, scales = gpu.glu_gated_linear(t["x"], t["w"], b, save=save, **p)
    close("h beside what is kept", h2, h, eh)
    if save == "bf16":
        kg, ku = ref.widened(pre, scales, N)
        for name, v, e, k, b16 in (("gate", g, eg, kg, pre[:, :N]), ("up", u, eu, ku, pre[:, N:])):
            # 12 significant bits, and BF16 the nearest to that (2^-8 of it at most)
            assert ((k - v).abs() <= 2.0 ** -12 * v.abs() + 1.01 * e + 2.0 ** -120).all(), name
            assert ((b16.to(D) - k).abs() <= BF16_HALF_ULP * k.abs() + 2.0 ** -120).all(), name
    else:
        # the codes are those of BF16 values within rounding of the exact ones
        kg, ku = ref.restored(pre, scales, N)
        NB = (N + 31) // 32
        for name, v, e, k, sc in (("gate", g, eg, kg, scales[:, :NB]), ("up", u, eu, ku, scales[:, NB:])):
            e = e + BF16_HALF_ULP * (1 + 2.0 ** -6) * v.abs()
            pad = lambda z: torch.nn.functional.pad(z, (0, -N % 32)).unflatten(1, (-1, 32)).amax(2)  # noqa: E731
            low, high = ref.mx_scale(pad(v.abs() - e).clamp(min=0)), ref.mx_scale(pad(v.abs() + e))
            assert ((sc >= low) & (sc <= high)).all(), name + " scales"
            step = torch.exp2(sc.to(D) - 127.0).repeat_interleave(32, 1)[:, :N]
            assert ((k - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -10 * step + 1.07 * e).all(), name + " codes"
    got = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, scales, bias=True, need_h=True, **p)
    want = ref.backward(t["dh"], t["x"], t["w"], kg, ku, act, layout, offsets)
    for name, a, terms in zip(("dx", "dw", "db"), got, (2 * N, M, M)):
        v, s, e = want[name]
        assert_close(name, a, v, s, terms + 8, e)
    hk = ref.act(kg.to(D), act) * ku.to(D)
    close("h again", got[3], hk, ref.rounding(kg.to(D), act) * (kg.to(D) * ku.to(D)).abs() + 2.0 ** -22 * hk.abs())
    return plain, h2, pre, scales, *got


# one row, few rows, each tile size and their edges; sums split, ragged and shorter than a step
SHAPES = [(1, 8, 8), (1, 24, 16), (2, 16, 72), (8, 520, 1032), (9, 40, 128), (17, 136, 1032), (33, 512, 64),
          (64, 248, 2048), (65, 64, 64), (100, 1000, 200), (128, 128, 136), (300, 520, 1096), (511, 72, 4104),
          (777, 1032, 520), (2500, 1032, 328), (3000, 2048, 64), (4000, 2008, 520)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("save", ["bf16", "mxfp8"])
def test_shapes(gpu, M, N, K, save):
    check(gpu, draw(M, N, K, seed=M + N), save=save, layout="paired" if M % 2 else "split")


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 64, 264), (20, 520, 2056), (200, 264, 512), (2300, 1160, 264)])
@pytest.mark.parametrize("layout", ["split", "paired"])
def test_activations(gpu, act, M, N, K, layout):
    for save in ("bf16", "mxfp8"):
        check(gpu, draw(M, N, K, seed=N), act, layout, save)
    check(gpu, draw(M, N, K, seed=N + 1), act, layout, "none", bias=False)


GROUPS = [([40, 50, 60], 0), ([0, 130, 0, 0, 257, 1, 0], 0), ([300, 0], 0), ([5, 0, 17, 64, 65, 3], 0), ([1] * 70, 0),
          ([2, 0, 1] * 43, 7), ([100, 200], 150), ([0, 0, 0], 40), ([0], 0), ([1500, 1, 1300, 900], 0)]


@pytest.mark.parametrize("counts,after", GROUPS, ids=[str(i) for i in range(len(GROUPS))])
@pytest.mark.parametrize("N,K,save", [(136, 200, "bf16"), (72, 1032, "mxfp8"), (264, 64, "mxfp8")])
def test_groups(gpu, counts, after, N, K, save):
    M = sum(counts) + after
    t = draw(M, N, K, groups=len(counts), seed=M)
    if after:                                    # rows of no group: whatever they hold, zeros come out
        t["x"][M - after:] = float("nan")
        t["dh"][M - after:] = float("inf")
        t["dh"] = t["dh"].clone()
    off = offsets_of(counts)
    x, t["x"] = t["x"], t["x"].nan_to_num(0.0)   # the reference sees zeros there
    kept = {}
    for layout in ("split", "paired"):
        p = dict(act="geglu", w_layout=layout, offsets=off)
        h, pre, scales = gpu.glu_gated_linear(x, t["w"], t["bias"], save=save, **p)
        _, _, (want, err) = ref.forward(t["x"], t["w"], t["bias"], "geglu", layout, off)
        want[M - after:], err[M - after:] = 0.0, 0.0
        close("h", h, want, err)
        dx, dw, db, again = gpu.glu_gated_linear_bwd(t["dh"], x, t["w"], pre, scales, bias=True, need_h=True, **p)
        kg, ku = ref.widened(pre, scales, N) if save == "bf16" else ref.restored(pre, scales, N)
        d0 = t["dh"].nan_to_num(0.0, 0.0, 0.0)
        ref_bwd = ref.backward(d0, t["x"], t["w"], kg, ku, "geglu", layout, off)
        for name, a, terms in zip(("dx", "dw", "db"), (dx, dw, db), (2 * N, M, M)):
            v, s, e = ref_bwd[name]
            assert_close(name, a, v, s, terms + 8, e)
        if after:
            assert (h[M - after:] == 0).all() and (dx[M - after:] == 0).all() and (again[M - after:] == 0).all()
            assert (pre[M - after:] == 0).all()
        kept[layout] = again
    assert all(torch.isfinite(v.float()).all() for v in kept.values())


@pytest.mark.parametrize("M,N,K", [(3, 72, 136), (150, 136, 264), (2100, 1160, 72)])
def test_strides(gpu, M, N, K):
    t = draw(M, N, K, ld=24)
    check(gpu, t)
    out = torch.full((M, N + 8), 7.0, dtype=BF16, device="cuda")
    h = gpu.glu_gated_linear(t["x"], t["w"], out=out[:, :N])
    assert (out[:, N:] == 7.0).all() and torch.equal(h, gpu.glu_gated_linear(t["x"], t["w"]))


def test_the_two_layouts_agree(gpu):
    for M in (1, 7, 40, 300, 3000):
        t = draw(M, 520, 328, seed=M)
        g, u = t["w"].chunk(2)
        bg, bu = t["bias"].chunk(2)
        w, b = torch.stack([g, u], 1).flatten(0, 1).contiguous(), torch.stack([bg, bu], 1).flatten().contiguous()
        for save in ("bf16", "mxfp8"):
            one = gpu.glu_gated_linear(t["x"], t["w"], t["bias"], save=save)
            two = gpu.glu_gated_linear(t["x"], w, b, w_layout="paired", save=save)
            assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_lengths_of_zero(gpu):
    t = draw(0, 64, 72)
    h, pre, scales = gpu.glu_gated_linear(t["x"], t["w"], t["bias"], save="mxfp8")
    assert h.shape == (0, 64) and pre.shape == (0, 128) and scales.shape == (0, 4)
    dx, dw, db, again = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, scales, bias=True, need_h=True)
    assert dx.shape == (0, 72) and (dw == 0).all() and (db == 0).all() and again.shape == (0, 64)
    for M in (5, 200):                           # a sum of no terms: the biases alone
        check(gpu, draw(M, 64, 0))
        t = draw(M, 0, 64)
        h, pre, _ = gpu.glu_gated_linear(t["x"], t["w"], save="bf16")
        assert h.shape == (M, 0)
        dx, dw, db, _ = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, bias=True)
        assert (dx == 0).all() and dw.shape == (0, 64) and db.shape == (0,)


def test_bf16_values_alone(gpu):
    """Gate and up from elsewhere, without the four bits."""
    t = draw(130, 72, 136)
    pre = (torch.randn(130, 144, device="cuda") * 2).to(BF16)
    got = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, bias=True, need_h=True)
    same = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, torch.zeros(130, 72, dtype=torch.uint8, device="cuda"),
                                    bias=True, need_h=True)
    assert all(torch.equal(a, b) for a, b in zip(got, same))
    da, db = gpu.glu_bwd(pre[:, :72], pre[:, 72:], t["dh"])
    dx, dw, _ = gpu.glu_linear_bwd(torch.cat([da, db], 1), t["x"], t["w"])
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    assert torch.equal(got[3], gpu.glu_fwd(pre[:, :72], pre[:, 72:]))


def test_only_what_is_wanted(gpu):
    t = draw(130, 72, 136)
    h, pre, scales = gpu.glu_gated_linear(t["x"], t["w"], save="mxfp8")
    full = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, scales, bias=True, need_h=True)
    for need in range(16):
        dx, dw, db, hh = (bool(need >> i & 1) for i in range(4))
        part = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, scales, need_dx=dx, need_dw=dw, bias=db, need_h=hh)
        for a, b, n in zip(part, full, (dx, dw, db, hh)):
            assert torch.equal(a, b) if n else a.numel() == 0


def test_large_pre_activations(gpu):
    """Gates in the tails of every activation."""
    t = draw(70, 136, 72, seed=9)
    for scale in (1.0, 8.0, 40.0, 2.0 ** 40):
        s = dict(t, x=(t["x"] * scale).to(BF16))
        for act in ref.ACTS:
            if scale > 100 and act != "swiglu":
                continue
            h = gpu.glu_gated_linear(s["x"], s["w"], act=act)
            _, _, (want, err) = ref.forward(s["x"], s["w"], None, act, "split")
            tol = BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err + 2.0 ** -120
            assert ((h.to(D) - want).abs() <= tol).all(), (act, scale)

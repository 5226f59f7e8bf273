"""8-bit products whose scales are near the ends of their range: the product of two scales may pass FP32's range
where the result does not.  One product of codes in the first block of the sum, small integers in the second, so
that every result is exact before its rounding."""
import pytest
import torch

from fp8_reference import E4M3, values
from ffn_reference import D

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def pick(g, choices, *shape):
    c = torch.tensor(choices, device="cuda")
    return c[torch.randint(0, len(choices), shape, generator=g, device="cuda")]


def code(t):
    return t.to(E4M3).view(torch.uint8)


# up to 8 rows; each tile size; a sum in parts
SHAPES = [(3, 136, 256, None), (8, 24, 4096, None), (40, 136, 256, None), (300, 264, 16384, None), (4000, 2008, 512, None),
          (2500, 1032, 256, None), (4096, 4096, 256, None), (4096, 4104, 256, None), (40, 136, 256, [0, 8, 8, 30, 38]),
          (700, 264, 256, [5, 300, 690])]


@pytest.mark.parametrize("M,N,K,offsets", SHAPES)
@pytest.mark.parametrize("w_scales", ["block", "row"])
@pytest.mark.parametrize("power", [70, -50])
def test_scales(gpu, M, N, K, offsets, w_scales, power):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    groups = 1 if offsets is None else len(offsets) - 1
    kb, least = K // 128, 2.0 ** -9
    x, w = torch.zeros(M, K, device="cuda"), torch.zeros(groups, N, K, device="cuda")
    w[..., :128] = pick(g, [0.0, 1.0, -448.0], groups, N, 128)
    x[:, 5], w[..., 5] = pick(g, [0.0, 0.0, least, -least, 1.0, 448.0], M), pick(g, [0.0, least, -3 * least, 1.0], groups, N)
    x[:, 128:256], w[..., 128:256] = pick(g, [0.0, 1.0, -1.0], M, 128), pick(g, [0.0, 1.0, 2.0], groups, N, 128)
    xs, nb = torch.ones(kb, M, device="cuda"), (N + 127) // 128
    ws = torch.ones((groups, nb, kb) if w_scales == "block" else (groups, kb, N), device="cuda")
    xs[0] = pick(g, [2.0 ** power, 2.0 ** (power + 4), 2.0 ** (2 * power - 22), 1.0], M)
    first = pick(g, [2.0 ** power, 1.0, 2.0 ** (power - 20)], *((groups, nb) if w_scales == "block" else (groups, N)))
    if w_scales == "block":
        ws[:, :, 0] = first
        wide = first.repeat_interleave(128, 1)[:, :N]
    else:
        ws[:, 0] = wide = first
    bad = M // 3
    xs[1, bad] = float("nan")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    args = (code(w), ws) if offsets is not None else (code(w[0]), ws[0])
    y = gpu.glu_linear_fp8(code(x), xs, *args, w_scales=w_scales, offsets=off)
    want = torch.zeros(M, N, dtype=F32, device="cuda")
    for e in range(groups):
        r = slice(0, M) if offsets is None else slice(offsets[e], offsets[e + 1])
        p = values(code(x[r, 5]))[:, None] * values(code(w[e, :, 5]))
        s = xs[0, r].to(D)[:, None] * wide[e].to(D)
        want[r] = (p * s + (x[r, 128:256] @ w[e, :, 128:256].t()).to(D)).to(F32)
    inside = offsets is None or offsets[0] <= bad < offsets[-1]
    if inside:
        want[bad] = float("nan")
    keep = ~torch.isnan(want)
    assert torch.equal(torch.isnan(y), ~keep)
    got, want = y[keep], want.to(BF16)[keep]
    # a product of two scales below 2^-126 is one of FP32's subnormal numbers
    if power > 0:
        assert torch.equal(got, want)
        assert M < 4096 or w_scales == "block" or (torch.isinf(want).any() and (want == 0).any())   # few scales: perhaps neither
    else:
        assert ((got.to(D) - want.to(D)).abs() <= 2.0 ** -124 + 2.0 ** -8 * want.to(D).abs()).all()


@pytest.mark.parametrize("M,N,K,offsets", SHAPES)
@pytest.mark.parametrize("w_scales", ["block", "row"])
def test_zero_and_small_sums_of_large_scales(gpu, M, N, K, offsets, w_scales):
    """Scales whose product is 2^140: sums of the first block are zero in the even rows and 2^-18, the least product of
    two codes, in the odd ones; the second block adds 1 times its scales, 1."""
    groups, kb = 1 if offsets is None else len(offsets) - 1, K // 128
    x, w = torch.zeros(M, K, device="cuda"), torch.zeros(groups, N, K, device="cuda")
    x[1::2, 100] = w[..., 100] = 2.0 ** -9
    w[..., 7] = 448.0
    x[:, 200] = w[..., 200] = 1.0
    xs = torch.ones(kb, M, device="cuda")
    ws = torch.ones((groups, (N + 127) // 128, kb) if w_scales == "block" else (groups, kb, N), device="cuda")
    xs[0] = 2.0 ** 70
    (ws[:, :, 0] if w_scales == "block" else ws[:, 0])[:] = 2.0 ** 70
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    args = (code(w), ws) if offsets is not None else (code(w[0]), ws[0])
    y = gpu.glu_linear_fp8(code(x), xs, *args, w_scales=w_scales, offsets=off)
    a, b = (0, M) if offsets is None else (offsets[0], offsets[-1])
    row = torch.arange(M, device="cuda")
    want = torch.where(row % 2 == 0, 1.0, 2.0 ** 122)
    want[:a], want[b:] = 0.0, 0.0
    assert torch.equal(y, want.to(BF16)[:, None].expand(M, N))

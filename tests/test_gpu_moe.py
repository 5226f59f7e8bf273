"""Expert routing on the GPU: places equal to a walk over the choices in order, copies to the byte,
weighted sums and gradients against 64 bits (ffn_reference.py)."""
import pytest
import torch

import ffn_reference as ref
from ffn_reference import assert_close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def choices(T, k, E, drop=0.0, skew=0.0, seed=0, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    ids = (torch.rand(T, k, generator=g) ** (1.0 + skew) * E).long().clamp(max=E - 1)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids.to(dtype)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 4), (3, 2, 300), (100, 4, 16), (1024, 1, 7), (1025, 1, 8),
                                   (700, 8, 64), (5000, 6, 60), (40000, 8, 256), (70000, 1, 1024), (30000, 3, 1000)])
@pytest.mark.parametrize("drop,skew", [(0.0, 0.0), (0.3, 4.0)])
def test_sort(gpu, T, k, E, drop, skew):
    ids = choices(T, k, E, drop, skew, seed=T)
    rows, offsets = gpu.glu_moe_sort(ids.cuda(), E)
    want_rows, want_offsets = ref.moe_sort(ids, E)
    assert torch.equal(rows.cpu(), want_rows) and torch.equal(offsets.cpu(), want_offsets)
    rows64, offsets64 = gpu.glu_moe_sort(ids.long().cuda(), E)
    assert torch.equal(rows64, rows) and torch.equal(offsets64, offsets)


def test_sort_numbers_outside_the_experts(gpu):
    ids = torch.tensor([[5, 1 << 40, 0], [-1, 4, -(1 << 40)], [(1 << 32) + 2, 2, 4]])
    rows, offsets = gpu.glu_moe_sort(ids.cuda(), 5)
    assert rows.tolist() == [[-1, -1, 0], [-1, 2, -1], [-1, 1, 3]] and offsets.tolist() == [0, 1, 1, 2, 2, 4]
    rows, offsets = gpu.glu_moe_sort(torch.full((3000, 2), -1, dtype=torch.int32, device="cuda"), 3)
    assert (rows == -1).all() and offsets.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("T,k", [(0, 4), (4, 0), (0, 0)])
def test_lengths_of_zero(gpu, T, k):
    rows, offsets = gpu.glu_moe_sort(torch.empty((T, k), dtype=torch.int32, device="cuda"), 6)
    assert rows.shape == (T, k) and offsets.tolist() == [0] * 7
    x = torch.randn(T, 40, device="cuda").to(BF16)
    xs = gpu.glu_moe_permute(x, rows, offsets)
    assert xs.shape == (0, 40)
    w = torch.empty((T, k), device="cuda")
    res = torch.randn(T, 40, device="cuda").to(BF16)
    assert torch.equal(gpu.glu_moe_combine(xs, rows, w, res), res)
    assert (gpu.glu_moe_combine(xs, rows) == 0).all()
    dy, dw = gpu.glu_moe_combine_bwd(res, xs, rows, w, offsets)
    assert dy.shape == (0, 40) and dw.shape == (T, k)


SHAPES = [(1, 1, 8, 3), (4, 8, 2048, 64), (37, 2, 100, 5), (300, 6, 1024, 60), (129, 9, 2056, 16), (50, 17, 333, 8),
          (513, 4, 7168, 32)]


def routed(gpu, T, k, H, E, drop, ld=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = choices(T, k, E, drop, 1.0, seed).cuda()
    rows, offsets = gpu.glu_moe_sort(ids, E)

    def n(rows_, scale=1.0):
        return (torch.randn((rows_, H + ld), generator=g, device="cuda") * scale).to(BF16)[:, :H]

    w = torch.rand((T, k), generator=g, device="cuda")
    return dict(rows=rows, offsets=offsets, x=n(T), y=n(T * k), w=w, res=n(T), dout=n(T, 0.1))


@pytest.mark.parametrize("T,k,H,E", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
def test_there_and_back(gpu, T, k, H, E, drop):
    t = routed(gpu, T, k, H, E, drop, seed=T)
    check(gpu, t, T, k, H)


@pytest.mark.parametrize("ld", [8, 3])
def test_strides(gpu, ld):
    check(gpu, routed(gpu, 60, 3, 520, 7, 0.1, ld=ld), 60, 3, 520)


def check(gpu, t, T, k, H):
    D = torch.float64
    rows, used = t["rows"].long(), int(t["offsets"][-1])
    live = rows >= 0
    src = torch.arange(T, device="cuda").unsqueeze(1).expand(T, k)[live]
    xs = gpu.glu_moe_permute(t["x"], t["rows"], t["offsets"])
    want = torch.zeros(T * k, H, dtype=BF16, device="cuda")
    want[rows[live]] = t["x"][src]
    assert torch.equal(xs.view(torch.int16), want.view(torch.int16))
    # what the rows of no expert hold is not read
    y = t["y"].clone()
    y[used:] = float("nan")
    picked = torch.where(live.unsqueeze(2), y[rows.clamp(min=0)].to(D).nan_to_num(), 0.0)
    for w, r in ((t["w"], t["res"]), (t["w"], None), (None, None)):
        out = gpu.glu_moe_combine(y, t["rows"], w, r)
        terms = picked * (w.to(D) if w is not None else torch.ones_like(t["w"], dtype=D)).unsqueeze(2)
        value, scale = terms.sum(1), terms.abs().sum(1)
        if r is not None:
            value, scale = value + r.to(D), scale + r.to(D).abs()
        assert_close("out", out, value, scale, k + 1)
    dy, dw = gpu.glu_moe_combine_bwd(t["dout"], y, t["rows"], t["w"], t["offsets"])
    d = t["dout"].to(D)
    want = torch.zeros(T * k, H, dtype=D, device="cuda")
    want[rows[live]] = t["w"].to(D)[live].unsqueeze(1) * d[src]
    assert_close("dy", dy, want, want.abs(), 1)
    prod = picked * d.unsqueeze(1)
    assert_close("dweights", dw, prod.sum(2), prod.abs().sum(2), H)
    assert (dw[~live] == 0).all() and (dy[used:] == 0).all()
    # the sum with ones is the gradient of the copy: <combine(a), b> = <a, permute(b)>
    a, b = gpu.glu_moe_combine(y, t["rows"]).to(D), t["x"].to(D)
    left = (a * b).sum()
    right = (torch.nan_to_num(y[:used].to(D)) * xs[:used].to(D)).sum()
    assert (left - right).abs() <= ref.BF16_HALF_ULP * (a * b).abs().sum() + 2.0 ** -20 * (
        y[:used].to(D) * xs[:used].to(D)).abs().sum()


@pytest.mark.parametrize("dtype,H", [(torch.uint8, 1), (torch.uint8, 33), (torch.uint8, 224), (torch.float32, 7),
                                     (torch.float64, 65), (torch.bfloat16, 5000), (torch.uint8, 7168)])
def test_permute_any_type(gpu, dtype, H):
    t = routed(gpu, 91, 3, 8, 6, 0.2)
    x = (torch.randn(91, H, device="cuda") * 50).to(dtype)
    xs = gpu.glu_moe_permute(x, t["rows"], t["offsets"])
    want = torch.zeros(91 * 3, H, dtype=dtype, device="cuda")
    live = t["rows"] >= 0
    want[t["rows"].long()[live]] = x[torch.arange(91, device="cuda").unsqueeze(1).expand(91, 3)[live]]
    assert torch.equal(xs, want)


def test_weights_gradient_against_differences(gpu):
    """dweights and dy along random directions against differences of the weighted sum in 64 bits (it is
    linear in each, so a difference of any size is exact)."""
    t = routed(gpu, 40, 4, 264, 9, 0.2)
    D = torch.float64
    dy, dw = gpu.glu_moe_combine_bwd(t["dout"], t["y"], t["rows"], t["w"], t["offsets"])
    live = (t["rows"] >= 0).to(D)

    def loss(y, w):
        return ((y[t["rows"].long().clamp(min=0)] * (w * live).unsqueeze(2)).sum(1) * t["dout"].to(D)).sum()

    y, w = t["y"].to(D), t["w"].to(D)
    v, u = torch.randn_like(w), torch.randn_like(y)
    a, b = loss(y, w + v) - loss(y, w), (dw.to(D) * v).sum()
    assert (a - b).abs() <= 264 * 2.0 ** -23 * (y.abs().max() * t["dout"].to(D).abs().sum() * v.abs().max() * 4)
    a, b = loss(y + u, w) - loss(y, w), (dy.to(D) * u).sum()
    assert (a - b).abs() <= ref.BF16_HALF_ULP * (dy.to(D) * u).abs().sum() * 1.02


def test_same_bits_again_and_on_another_stream(gpu):
    t = routed(gpu, 3000, 6, 520, 40, 0.1)
    ids = choices(3000, 6, 40, 0.1, 1.0).cuda()

    def run():
        rows, offsets = gpu.glu_moe_sort(ids, 40)
        return (rows, offsets, gpu.glu_moe_permute(t["x"], rows, offsets), gpu.glu_moe_combine(t["y"], rows, t["w"])) \
            + gpu.glu_moe_combine_bwd(t["dout"], t["y"], rows, t["w"], offsets)

    a = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_offsets_past_32_bits(gpu):
    """33000 tokens of 8 choices and 8704 columns: the sorted rows take 4.6 GB."""
    T, k, H, E = 33000, 8, 8704, 16
    t = routed(gpu, T, k, 8, E, 0.0)
    x = torch.randn(T, H, device="cuda", dtype=BF16)
    xs = gpu.glu_moe_permute(x, t["rows"], t["offsets"])
    pick = torch.tensor([0, 1, 777, T - 1], device="cuda")
    for j in range(k):
        assert torch.equal(xs[t["rows"][pick, j].long()], x[pick])
    out = gpu.glu_moe_combine(xs, t["rows"], t["w"])
    want = x[pick].double() * t["w"][pick].double().sum(1, keepdim=True)
    assert_close("out", out[pick], want, want.abs(), 2 * k)
    dy, dw = gpu.glu_moe_combine_bwd(x, xs, t["rows"], t["w"], t["offsets"])
    sq = x[pick].double().square().sum(1, keepdim=True).expand(-1, k)
    assert_close("dweights", dw[pick], sq, sq, H)
    for j in range(k):
        want = x[pick].double() * t["w"][pick, j].double().unsqueeze(1)
        assert_close("dy", dy[t["rows"][pick, j].long()], want, want.abs(), 1)

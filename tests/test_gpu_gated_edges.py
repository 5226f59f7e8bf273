"""The gated projections, the checkpoints and the 8-bit products where they can go wrong: captured and
replayed, on other streams, two calls at once, past 32-bit offsets, NaN and infinities, gradients
against differences."""
import pytest
import torch

import fp8_reference as fref
import gated_reference as ref
from ffn_reference import BF16_HALF_ULP, D, assert_close

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def n(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def operands(M=300, N=72, K=4096, groups=None, seed=0):
    lead = () if groups is None else (groups,)
    off = None
    if groups is not None:
        off = torch.arange(0, groups + 1, device="cuda", dtype=torch.int32) * (M // groups)
    return dict(x=n(M, K, seed=seed), w=n(*lead, 2 * N, K, seed=seed + 1, scale=K ** -0.5), b=n(*lead, 2 * N, seed=seed + 2),
                dh=n(M, N, seed=seed + 3, scale=0.1), w2=n(*lead, 136, N, seed=seed + 4, scale=N ** -0.5), off=off)


def everything(gpu, t):
    """One call of each entry point, and what it returns."""
    out = []
    for save in ("bf16", "mxfp8"):
        h, pre, extra = gpu.glu_gated_linear(t["x"], t["w"], t["b"], offsets=t["off"], save=save)
        out += [h, pre, extra, *gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, extra, offsets=t["off"], bias=True,
                                                         need_h=True)]
    h, q, s = gpu.glu_fwd_ckpt(h, t["dh"])
    out += [h, q, s, *gpu.glu_bwd_ckpt(q, s, t["dh"], need_h=True)]
    q_row, q_col, s_row, s_col = gpu.glu_quant_fp8(t["x"], colwise=True)
    wq, ws, wt, wts = gpu.glu_quant_fp8_weight(t["w"], transpose=True)
    out += [q_row, q_col, s_row, s_col, wq, ws, wt, wts]
    out += [gpu.glu_linear_fp8(q_row, s_row, wq, ws, t["b"], offsets=t["off"])]
    hq, _, hs, _ = gpu.glu_fwd_fp8(h, t["dh"])
    w2q, w2s, _, _ = gpu.glu_quant_fp8_weight(t["w2"])
    return out + [hq, hs, gpu.glu_linear_fp8(hq, hs, w2q, w2s, offsets=t["off"])]


def bits(t):
    return t.contiguous().view(torch.uint8) if t.numel() else t


def same(a, b):
    return [i for i, (u, v) in enumerate(zip(a, b)) if not torch.equal(bits(u), bits(v))]


CALLS = [dict(), dict(M=5, N=520), dict(M=40, K=272), dict(M=2600, N=520, K=144), dict(groups=3, K=272),
         dict(M=24, groups=12, K=272)]


@pytest.mark.parametrize("kw", CALLS, ids=[str(i) for i in range(len(CALLS))])
def test_same_bits_again_and_on_another_stream(gpu, kw):
    t = operands(**kw)
    a = everything(gpu, t)
    assert not same(a, everything(gpu, t))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = everything(gpu, t)
    torch.cuda.current_stream().wait_stream(s)
    assert not same(a, b)


def test_two_calls_at_once(gpu):
    t, u = operands(seed=1), operands(M=513, N=136, K=1040, seed=2)
    want = everything(gpu, t), everything(gpu, u)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, (s, v) in enumerate(zip(streams, (t, u))):
            with torch.cuda.stream(s):
                got[i] = everything(gpu, v)
        torch.cuda.synchronize()
        assert not same(want[0], got[0]) and not same(want[1], got[1])


@pytest.mark.parametrize("kw", CALLS, ids=[str(i) for i in range(len(CALLS))])
def test_captured_and_replayed(gpu, kw):
    t = operands(**kw)
    want = everything(gpu, t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = everything(gpu, t)
    x, other = t["x"].clone(), operands(**kw, seed=50)
    for turn in range(4):
        for o in out:
            o.view(torch.uint8).fill_(0xA5 if turn % 2 else 0) if o.numel() else None
        if turn == 2:                              # other values in the same place, and back
            t["x"].copy_(other["x"])
            g.replay()
            torch.cuda.synchronize()
            assert not same(everything(gpu, t), out)
            t["x"].copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert not same(want, out)
        everything(gpu, other)                     # eager work in between
        torch.cuda.synchronize()


def test_two_captured_graphs(gpu):
    """Graphs of two calls replayed in turn and at once: no scratch memory in common."""
    t, u = operands(seed=3), operands(M=513, N=136, K=1040, seed=4)
    want = everything(gpu, t), everything(gpu, u)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for v in (t, u):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(gpu, v))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert not same(want[0], outs[0]) and not same(want[1], outs[1])


def test_nan_stays_in_its_row(gpu):
    for M in (3, 40, 300, 2600):
        t = operands(M=M, N=136, K=264, seed=M)
        for save in ("bf16", "mxfp8"):
            a = gpu.glu_gated_linear(t["x"], t["w"], t["b"], save=save)
            ga = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], *a[1:], need_h=True)
            x = t["x"].clone()
            x[1, 3] = float("nan")
            b = gpu.glu_gated_linear(x, t["w"], t["b"], save=save)
            gb = gpu.glu_gated_linear_bwd(t["dh"], x, t["w"], *b[1:], need_h=True)
            keep = torch.arange(M, device="cuda") != 1
            for u, v in zip(a, b):
                assert torch.equal(u[keep], v[keep])
            assert torch.isnan(b[0][1]).all() and torch.isnan(gb[0][1]).all() and torch.isnan(gb[3][1]).all()
            assert torch.equal(ga[0][keep], gb[0][keep]) and torch.equal(ga[3][keep], gb[3][keep])


def test_infinite_pre_activations(gpu):
    """Sums that leave FP32's range stay what they are: kept as infinities and NaN, never as finite values."""
    t = operands(M=40, N=72, K=264)
    x = t["x"].clone()
    x[5] = torch.where(x[5] < 0, -3e38, 3e38).to(BF16)
    w = t["w"].abs()
    h, pre, extra = gpu.glu_gated_linear(x, w, save="bf16")
    g, u = ref.widened(pre, extra, 72)
    exact = x[5].double() @ w.double().t()
    over = exact.abs() > 4e38
    got = torch.cat([g[5], u[5]])
    assert not torch.isfinite(got[over]).any()
    _, codes, scales = gpu.glu_gated_linear(x, w, save="mxfp8")
    assert torch.equal(torch.isnan(torch.cat(ref.restored(codes, scales, 72), 1))[:5],
                       torch.zeros(5, 144, dtype=torch.bool, device="cuda"))


def test_offsets_past_32_bits(gpu):
    """The up half of W more than 2^31 bytes behind the gate half, for few and for many rows; rows past 2^31
    bytes of every operand."""
    N, K = 135168, 8200
    w = torch.zeros(2 * N, K, device="cuda", dtype=BF16)
    cols = torch.tensor([0, 1, 7, 31, 32, 1000, N // 2, N - 33, N - 8, N - 1], device="cuda")
    w[cols] = n(10, K, seed=1, scale=K ** -0.5)
    w[N + cols] = n(10, K, seed=2, scale=K ** -0.5)
    small = torch.cat([w[cols], w[N + cols]])
    for M in (3, 20, 200):
        x = n(M, K, seed=M)
        h = gpu.glu_gated_linear(x, w)
        _, _, (want, err) = ref.forward(x, small, None, "swiglu", "split")
        assert ((h[:, cols].to(D) - want).abs() <= BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err + 2.0 ** -120).all()
        h[:, cols] = 0
        assert (h == 0).all()
    del w, h
    M, N, K, last = 1200000, 1032, 2056, 300
    x = torch.zeros(M, K, device="cuda", dtype=BF16)
    x[-last:] = n(last, K, seed=5)
    w, dh = n(2 * N, K, seed=6, scale=K ** -0.5), torch.zeros(M, N, device="cuda", dtype=BF16)
    dh[-last:] = n(last, N, seed=7)
    _, _, (want, err) = ref.forward(x[-last:], w, None, "swiglu", "split")
    for save in ("bf16", "mxfp8"):
        h, pre, extra = gpu.glu_gated_linear(x, w, save=save)
        assert (h[:-last] == 0).all() and (pre[:-last] == 0).all()
        assert ((h[-last:].to(D) - want).abs() <= BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err + 2.0 ** -120).all()
        kept = ref.widened(pre[-last:], extra[-last:], N) if save == "bf16" else ref.restored(pre[-last:], extra[-last:], N)
        dx, dw, db, again = gpu.glu_gated_linear_bwd(dh, x, w, pre, extra, bias=True, need_h=True)
        grads = ref.backward(dh[-last:], x[-last:], w, *kept, "swiglu", "split")
        assert (dx[:-last] == 0).all() and (again[:-last] == 0).all()
        for name, a, terms in (("dx", dx[-last:], 2 * N), ("dw", dw, 4096), ("db", db, 4096)):
            assert_close(name, a, *grads[name][:2], terms, grads[name][2])
        del h, pre, extra, dx, dw, db, again


def test_checkpoints_past_32_bits(gpu):
    M, N = 300000, 8200
    gate = torch.zeros(M, N, device="cuda", dtype=BF16)
    up = torch.ones(M, N, device="cuda", dtype=BF16)
    gate[-40:], up[-40:] = n(40, N, seed=1), n(40, N, seed=2)
    h, q, s = gpu.glu_fwd_ckpt(gate, up)
    same_rows = gpu.glu_fwd_ckpt(gate[-40:], up[-40:])
    for a, b in zip((h, q, s), same_rows):
        assert torch.equal(a[-40:], b)
    assert (h[:-40] == 0).all()
    d, again = gpu.glu_bwd_ckpt(q, s, up, need_h=True)
    e, f = gpu.glu_bwd_ckpt(*same_rows[1:], up[-40:], need_h=True)
    assert torch.equal(d[-40:], e) and torch.equal(again[-40:], f)


def test_8_bit_products_past_32_bits(gpu):
    M, N, K, last = 1200000, 72, 2064, 300
    x = torch.zeros(M, K, device="cuda", dtype=BF16)
    x[-last:] = n(last, K, seed=1)
    q, qt, s, st = gpu.glu_quant_fp8(x, colwise=True)
    a, at, b, bt = gpu.glu_quant_fp8(x[-last:].contiguous(), colwise=True)
    assert torch.equal(q[-last:], a) and torch.equal(s[:, -last:], b) and (q[:-last] == 0).all()
    assert torch.equal(qt[:, M // 128 * 128:M], gpu.glu_quant_fp8(x[M // 128 * 128:], rowwise=False, colwise=True)[1][:, :M % 128])
    assert (qt[:, :M - last] == 0).all()
    w = n(N, K, seed=2, scale=K ** -0.5)
    wq, ws, _, _ = gpu.glu_quant_fp8_weight(w)
    y = gpu.glu_linear_fp8(q, s, wq, ws)
    want, err, _ = fref.product(a, b, wq, ws, "block")
    assert (y[:-last] == 0).all()
    assert ((y[-last:].to(D) - want).abs() <= BF16_HALF_ULP * want.abs() * (1 + 2.0 ** -6) + err).all()


def test_gradient_against_differences(gpu):
    """The gradients along random directions against central differences in 64 bits, with save="bf16"."""
    M, N, K = 40, 72, 136
    t = operands(M, N, K)
    for act in ref.ACTS:
        for layout in ("split", "paired"):
            h, pre, extra = gpu.glu_gated_linear(t["x"], t["w"], t["b"], act=act, w_layout=layout, save="bf16")
            grads = gpu.glu_gated_linear_bwd(t["dh"], t["x"], t["w"], pre, extra, act=act, w_layout=layout, bias=True)[:3]
            at = dict(x=t["x"].double(), w=t["w"].double(), b=t["b"].double())

            def loss(v):
                g, u = ref.halves(v["x"] @ v["w"].t() + v["b"], layout, 1)
                return (ref.act(g, act) * u * t["dh"].double()).sum()

            r = torch.Generator(device="cuda").manual_seed(5)
            for name, grad in zip(("x", "w", "b"), grads):
                v = torch.randn(grad.shape, generator=r, device="cuda", dtype=D)
                e = 1e-5
                lo, hi = (loss({**at, name: at[name] + d * v}) for d in (-e, e))
                slope, dot = (hi - lo) / (2 * e), (grad.double() * v).sum()
                # each element is off by its own rounding, dp's, and what 12 bits of gate and up leave open
                tol = 3 * BF16_HALF_ULP * (grad.double() * v).abs().sum()
                assert (slope - dot).abs() <= tol, (act, layout, name, slope.item(), dot.item(), tol.item())

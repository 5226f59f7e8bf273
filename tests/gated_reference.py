"""Plain 64-bit references of the gated projections and of MXFP8 checkpoints, with what an FP32
evaluation and the stated roundings may move (see ffn_reference.py)."""
import torch

from ffn_reference import ACT_ERROR, BF16_HALF_ULP, D, segments

ACTS = ("swiglu", "geglu", "geglu_erf", "relu2")


def act(g, name):
    F = torch.nn.functional
    return {"swiglu": F.silu, "geglu": lambda t: F.gelu(t, approximate="tanh"), "geglu_erf": F.gelu,
            "relu2": lambda t: F.relu(t).square()}[name](g)


def act_grad(g, name):
    g = g.detach().requires_grad_(True)
    return torch.autograd.grad(act(g, name).sum(), g)[0]


def steepest(g, name):
    """A bound on |act'| near g."""
    return 2.0 * g.abs() if name == "relu2" else torch.full_like(g, 1.13)


def rounding(g, name):
    """How far act and act' in FP32 may be off, over |g| and over 1: products alone for relu2."""
    return 2.0 ** -22 * (1.0 + g.abs()) if name == "relu2" else torch.full_like(g, ACT_ERROR)


def halves(t, layout, dim):
    n = t.shape[dim] // 2
    if layout == "split":
        return t.narrow(dim, 0, n), t.narrow(dim, n, n)
    t = t.movedim(dim, 0)
    return t[0::2].movedim(0, dim), t[1::2].movedim(0, dim)


def joined(a, b, layout):
    return torch.cat([a, b], 1) if layout == "split" else torch.stack([a, b], 2).flatten(1)


def forward(x, w, bias, name, layout, offsets=None):
    """(gate, error), (up, error) and (h, error) before the last rounding."""
    M, N, K = x.shape[0], w.shape[-2] // 2, x.shape[1]
    g, u, eg, eu = (torch.zeros(M, N, dtype=D, device=x.device) for _ in range(4))
    t = (K + 8) * 2.0 ** -23
    for e, a, b in segments(M, offsets):
        W = w if w.dim() == 2 else w[e]
        B = None if bias is None else (bias if w.dim() == 2 else bias[e])
        X = x[a:b].to(D)
        for out, err, part in ((g, eg, 0), (u, eu, 1)):
            Wp = halves(W, layout, 0)[part].to(D)
            out[a:b], err[a:b] = X @ Wp.t(), t * (X.abs() @ Wp.abs().t())
            if B is not None:
                Bp = halves(B, layout, 0)[part].to(D)
                out[a:b] += Bp
                err[a:b] += t * Bp.abs()
    A = act(g, name)
    eh = (steepest(g.abs() + eg, name) * eg + rounding(g, name) * g.abs()) * (u.abs() + eu) + A.abs() * eu
    return (g, eg), (u, eu), (A * u, eh + 2.0 ** -22 * (A * u).abs())


def backward(dh, x, w, gate, up, name, layout, offsets=None):
    """{name: (value, scale, extra)} from the gate and up values kept: extra is what act' in FP32 and
    dp rounded to BF16 (for the products, not for db) can move."""
    M, (N2, K) = x.shape[0], w.shape[-2:]
    G = w.shape[0] if w.dim() == 3 else 1
    g, u, d = gate.to(D), up.to(D), dh.to(D)
    dp = joined(d * u * act_grad(g, name), d * act(g, name), layout)
    off = joined((d * u).abs() * rounding(g, name), d.abs() * rounding(g, name) * g.abs(), layout) + 2.0 ** -22 * dp.abs()
    moved = off + BF16_HALF_ULP * dp.abs() + 2.0 ** -134
    zeros = lambda *n: torch.zeros(*n, dtype=D, device=x.device)  # noqa: E731
    out = {k: [zeros(*s) for _ in range(3)] for k, s in (("dx", (M, K)), ("dw", (G, N2, K)), ("db", (G, N2)))}
    for e, a, b in segments(M, offsets):
        W, X, p, m = (w if w.dim() == 2 else w[e]).to(D), x[a:b].to(D), dp[a:b], moved[a:b]
        for t, v in zip(out["dx"], (p @ W, p.abs() @ W.abs(), m @ W.abs())):
            t[a:b] = v
        for t, v in zip(out["dw"], (p.t() @ X, p.abs().t() @ X.abs(), m.t() @ X.abs())):
            t[e] = v
        for t, v in zip(out["db"], (p.sum(0), p.abs().sum(0), off[a:b].sum(0))):
            t[e] = v
    if w.dim() == 2:
        out.update(dw=[t[0] for t in out["dw"]], db=[t[0] for t in out["db"]])
    return out


def mx_scale(top):
    """The E8M0 byte of a block whose largest magnitude is `top` (64 bits): e + 127 for the least e
    with 448 2^e >= top."""
    e = torch.floor(torch.log2((top / 448.0).clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e) * 448.0 >= top, e, e + 1.0)
    return torch.where(torch.isfinite(top), e.clamp(min=-127.0) + 127.0, 255.0).to(torch.uint8)


def restored(q, s, N):
    """[gate, up] in 64 bits from codes [M, 2N] and scales [M, 2 ceil(N/32)]."""
    v = q.view(torch.float8_e4m3fn).to(D)
    NB, out = (N + 31) // 32, []
    for h in range(2):
        sc = s[:, h * NB:(h + 1) * NB].repeat_interleave(32, 1)[:, :N]
        f = torch.where(sc == 255, float("nan"), torch.exp2(sc.to(D) - 127.0))
        out.append(v[:, h * N:(h + 1) * N] * f)
    return out


def widened(pre, extra, N):
    """[gate, up] in 64 bits from BF16 [M, 2N] and the four more bits of each, [M, N] bytes."""
    nib = torch.stack([extra & 15, extra >> 4], 2).flatten(1).to(torch.int32)
    bits = pre.view(torch.int16).to(torch.int32) * 65536 + torch.where(nib > 7, nib - 16, nib) * 4096
    v = bits.view(torch.float32).to(D)
    return v[:, :N], v[:, N:]

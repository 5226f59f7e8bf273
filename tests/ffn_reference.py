"""Plain 64-bit references of the operators around the GLU, with the scale each result's
rounding errors are measured against.

A reference returns, for every output, the value from the definition and `scale`, the sum of
the magnitudes of the terms the value is formed from.  An FP32 evaluation of n terms is within
n 2^-23 of `scale` of the value, and a result rounded to BF16 (8 significant bits) moves by at
most 2^-8 of itself; `assert_close` asserts the sum of the two."""
import torch

D = torch.float64
BF16_HALF_ULP = 2.0 ** -8   # of the value: 8 significant bits, the worst just above a power of two
ACT_ERROR = 2.0 ** -18      # of act and act' in FP32: exp2, reciprocal and the erfc fit (7e-7), each to a few ulps


def half_ulp(t):
    return {torch.bfloat16: BF16_HALF_ULP, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[t.dtype]


def assert_close(name, got, ref, scale, terms, extra=0.0):
    """|got - ref| <= half an ulp of got's type + terms 2^-23 scale + extra, element by element
    (2^-120 more, for subnormal results)."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if got.numel() == 0:
        return
    tol = half_ulp(got) * ref.abs() * (1 + 2.0 ** -6) + terms * 2.0 ** -23 * scale + extra + 2.0 ** -120
    err = (got.to(D) - ref).abs()
    assert torch.isfinite(got.float()).all(), f"{name}: not finite"
    bad = err > tol
    if bad.any():
        i = int((err / tol).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: got "
                             f"{got.reshape(-1)[i].item()} for {ref.reshape(-1)[i].item()}, off by "
                             f"{err.reshape(-1)[i].item():.3g}, allowed {tol.reshape(-1)[i].item():.3g}")


# ---- norms -----------------------------------------------------------------------------------

def spread(p, M):
    """A parameter [H] or [G, H] as FP64, one row per row of x."""
    p = p.to(D)
    if p.dim() == 1:
        p = p.unsqueeze(0)
    return p.repeat_interleave(M // p.shape[0], 0) if p.shape[0] > 1 else p.expand(M, -1)


def normed(v, s, kind, eps):
    """(n, 1/sigma, scale of n) of the rows of v, whose own error scale is s."""
    if kind == "layer":
        m = v.mean(1, keepdim=True)
        s = s + s.mean(1, keepdim=True)
        v = v - m
    r = 1.0 / (v.square().mean(1, keepdim=True) + eps).sqrt()
    n = v * r
    # d(n) = r (dv - n mean(n dv)): the elements' errors, and that of the row's own sum
    return n, r, r * s + n.abs() * (1.0 + (r * s * n.abs()).mean(1, keepdim=True))


def norm_forward(x, y, gate=None, w_pre=None, b_pre=None, w_post=None, pre=True, post=False, res_scale=1.0,
                 kind="rms", eps=1e-6):
    """{name: (value, scale)} of x_out and h, and what the gradients need."""
    M = x.shape[0]
    X = x.to(D)
    c = dict(r={})
    if y is None:
        xo, s = X, X.abs()
    else:
        Y = y.to(D)
        ny, ry, sn = normed(Y, Y.abs(), kind, eps) if post else (Y, None, Y.abs())
        w = spread(w_post, M) if w_post is not None else torch.ones_like(Y)
        g = spread(gate, M) if gate is not None else torch.ones_like(Y)
        z, sz = ny * w, sn * w.abs()
        xo, s = res_scale * X + g * z, abs(res_scale) * X.abs() + g.abs() * sz
        c.update(ny=ny, ry=ry, sn=sn, w=w, g=g, z=z, sz=sz)
    out = dict(x_out=(xo, s))
    if pre:
        nx, rx, snx = normed(xo, s, kind, eps)
        wp = spread(w_pre, M) if w_pre is not None else torch.ones_like(X)
        h, sh = nx * wp, snx * wp.abs()
        if b_pre is not None:
            b = spread(b_pre, M)
            h, sh = h + b, sh + b.abs()
        out["h"] = (h, sh)
        c.update(nx=nx, rx=rx, snx=snx, wp=wp)
    return out, c


def norm_backward(x, y, dx_out, dh, gate=None, w_pre=None, b_pre=None, w_post=None, pre=True, post=False,
                  res_scale=1.0, kind="rms", eps=1e-6):
    """{name: (value, scale)} of every gradient, from the formulas."""
    M, H = x.shape
    _, c = norm_forward(x, y, gate, w_pre, b_pre, w_post, pre, post, res_scale, kind, eps)

    def through(dn, sdn, n, sn, r):
        """Gradient of v from that of n = N(v)."""
        lay = kind == "layer"
        g = dn - n * (dn * n).mean(1, keepdim=True) - (dn.mean(1, keepdim=True) if lay else 0)
        inner = (sdn * n.abs() + dn.abs() * sn).mean(1, keepdim=True)
        sg = sdn + sn * (dn * n).abs().mean(1, keepdim=True) + n.abs() * inner
        sg = sg + (sdn.mean(1, keepdim=True) if lay else 0)
        return g * r, 2.0 * sg * r

    def groups(t, p):
        G = 1 if p.dim() == 1 else p.shape[0]
        return t.reshape(G, M // G, H).sum(1).reshape(p.shape)

    out = {}
    Dv = dx_out.to(D) if dx_out is not None else torch.zeros(M, H, dtype=D, device=x.device)
    s = Dv.abs()
    if pre:
        d = dh.to(D)
        if w_pre is not None:
            out["dw_pre"] = (groups(d * c["nx"], w_pre), groups(d.abs() * c["snx"], w_pre))
        if b_pre is not None:
            out["db_pre"] = (groups(d, b_pre), groups(d.abs(), b_pre))
        g, sg = through(d * c["wp"], (d * c["wp"]).abs(), c["nx"], c["snx"], c["rx"])
        Dv, s = Dv + g, s + sg
    out["dx"] = (res_scale * Dv, abs(res_scale) * s)
    if y is not None:
        if gate is not None:
            out["dgate"] = (groups(Dv * c["z"], gate), groups(s * c["z"].abs() + Dv.abs() * c["sz"], gate))
        dz, sz = c["g"] * Dv, c["g"].abs() * s
        if w_post is not None:
            out["dw_post"] = ((dz * c["ny"]).sum(0), (sz * c["ny"].abs() + dz.abs() * c["sn"]).sum(0))
        if post:
            dz, sz = through(dz * c["w"], sz * c["w"].abs(), c["ny"], c["sn"], c["ry"])
        out["dy"] = (dz, sz)
    return out


# ---- linear products -------------------------------------------------------------------------

def act(p, name):
    F = torch.nn.functional
    return {"none": lambda t: t, "silu": F.silu, "gelu": lambda t: F.gelu(t, approximate="tanh"),
            "gelu_erf": F.gelu}[name](p)


def act_grad(p, name):
    p = p.detach().requires_grad_(True)
    return torch.autograd.grad(act(p, name).sum(), p)[0] if name != "none" else torch.ones_like(p)


def segments(M, offsets):
    """[(group, first row, past the last row)] and the rows of no group."""
    if offsets is None:
        return [(0, 0, M)]
    o = [min(max(v, 0), M) for v in offsets.tolist()]
    return [(e, o[e], max(o[e], o[e + 1])) for e in range(len(o) - 1)]


def linear_forward(x, w, bias=None, residual=None, act_name="none", offsets=None):
    """y and p (the pre-activation), each (value, scale, extra)."""
    M, N = x.shape[0], w.shape[-2]
    p, sp, y, sy = (torch.zeros(M, N, dtype=D, device=x.device) for _ in range(4))
    for e, a, b in segments(M, offsets):
        W = (w if w.dim() == 2 else w[e]).to(D)
        X = x[a:b].to(D)
        p[a:b], sp[a:b] = X @ W.t(), X.abs() @ W.abs().t()
        if bias is not None:
            t = (bias if w.dim() == 2 else bias[e]).to(D)
            p[a:b] += t
            sp[a:b] += t.abs()
        y[a:b], sy[a:b] = act(p[a:b], act_name), 1.13 * sp[a:b]   # |act'| <= 1.13
        if residual is not None:
            y[a:b] += residual[a:b].to(D)
            sy[a:b] += residual[a:b].to(D).abs()
    return (y, sy, ACT_ERROR * p.abs() if act_name != "none" else 0.0), (p, sp, 0.0)


def linear_backward(dy, x, w, pre, act_name="none", offsets=None):
    """{name: (value, scale, extra)} of dx, dw, db from the pre-activation `pre` as saved; extra is
    what act' in FP32 and dp rounded to BF16 (for the products, not for db) can move."""
    M, (N, K) = x.shape[0], w.shape[-2:]
    G = w.shape[0] if w.dim() == 3 else 1
    zeros = lambda *n: torch.zeros(*n, dtype=D, device=x.device)  # noqa: E731
    dx, sdx, edx = zeros(M, K), zeros(M, K), zeros(M, K)
    dw, sdw, edw = zeros(G, N, K), zeros(G, N, K), zeros(G, N, K)
    db, sdb, edb = zeros(G, N), zeros(G, N), zeros(G, N)
    for e, a, b in segments(M, offsets):
        W = (w if w.dim() == 2 else w[e]).to(D)
        X, d = x[a:b].to(D), dy[a:b].to(D)
        off = torch.zeros_like(d)
        if act_name != "none":
            off = ACT_ERROR * d.abs()
            d = d * act_grad(pre[a:b].to(D), act_name)
        moved = off + (BF16_HALF_ULP * d.abs() if act_name != "none" else 0.0)
        dx[a:b], sdx[a:b], edx[a:b] = d @ W, d.abs() @ W.abs(), moved @ W.abs()
        dw[e], sdw[e], edw[e] = d.t() @ X, d.abs().t() @ X.abs(), moved.t() @ X.abs()
        db[e], sdb[e], edb[e] = d.sum(0), d.abs().sum(0), off.sum(0)
    if w.dim() == 2:
        dw, sdw, edw, db, sdb, edb = (t[0] for t in (dw, sdw, edw, db, sdb, edb))
    return dict(dx=(dx, sdx, edx), dw=(dw, sdw, edw), db=(db, sdb, edb))


# ---- expert routing --------------------------------------------------------------------------

def moe_sort(ids, experts):
    """(rows, offsets) by walking the choices in order."""
    flat = ids.reshape(-1).tolist()
    queue = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            queue[e].append(i)
    rows, offsets, at = [-1] * len(flat), [0], 0
    for q in queue:
        for i in q:
            rows[i] = at
            at += 1
        offsets.append(at)
    return (torch.tensor(rows, dtype=torch.int32).reshape(ids.shape), torch.tensor(offsets, dtype=torch.int32))

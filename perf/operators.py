"""Cases that measure the operators around the GLU: the norms of a block, the linear products
(dense and per expert), and the routing of tokens to experts and back.

Three groups of operators, each in the forms a feed-forward block uses:

  norm     x' = res_scale x + gate * norm(y; w_post) and h = norm(x'; w_pre, b_pre), in one
           pass; with "train" also every gradient.
  linear   act(x W^T + b) + residual; with "train" also dx, dW, db.  "experts" > 0: row groups
           given by offsets, one W and b per group.
  moe      tokens sorted by expert, copied into that order and combined back with their
           weights; with "train" also the gradients of the copy and of the combination.

`own` selects between the plain form (elementary torch operations in FP32, rounded once at the
end) and the library's entry points.  A case is a dict of plain values; `prepare` makes the
tensors of a case from a seed, `run` is one pass, `exact` the same results in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
BF16, F32 = torch.bfloat16, torch.float32


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # one new token through the norms on both sides of a block: launch latency
        dict(name="norm-token", op="norm", M=1, H=2048, groups=1, kind="rms", dtype="bf16", post=True,
             train=False),
        # the rows of 8 requests with a gate, weight and shift per request (adaptive norm)
        dict(name="norm-adaptive", op="norm", M=968, H=2048, groups=8, kind="rms", dtype="bf16", post=False,
             train=False),
        # a training step at the library's large activation shape
        dict(name="norm-train", op="norm", M=16384, H=7168, groups=1, kind="rms", dtype="bf16", post=True,
             train=True),
        # a ragged width, LayerNorm, residual stream and parameters in FP32
        dict(name="norm-train-odd", op="norm", M=1021, H=8193, groups=1, kind="layer", dtype="f32", post=True,
             train=True),
        # the down projection for one new token: one pass over the weights
        dict(name="linear-token", op="linear", M=1, N=2048, K=16384, act="none", experts=0, train=False),
        # the same projection for a prefill of 968 rows: few output tiles, a long sum
        dict(name="linear-prefill", op="linear", M=968, N=2048, K=16384, act="none", experts=0, train=False),
        # a large training step with bias, GELU and residual
        dict(name="linear-train", op="linear", M=16384, N=7168, K=2048, act="gelu", experts=0, train=True),
        # a small ragged training step: no extent is a multiple of a tile
        dict(name="linear-train-odd", op="linear", M=1021, N=1000, K=2056, act="silu", experts=0, train=True),
        # a decoding step of 32 experts on 256 routed rows: every expert's weights, few rows each
        dict(name="experts-decode", op="linear", M=256, N=2048, K=2048, act="none", experts=32, train=False),
        # a training step of 16 experts
        dict(name="experts-train", op="linear", M=16384, N=4096, K=2048, act="none", experts=16, train=True),
        # four decoding tokens to their experts and back
        dict(name="moe-token", op="moe", T=4, k=8, E=64, H=2048, drop=0.0, train=False),
        # a training step's routing, some choices dropped by a capacity limit
        dict(name="moe-train", op="moe", T=8192, k=8, E=64, H=7168, drop=0.02, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "linear", "experts", "moe", "moe"))
    train = rng.random() < 0.5
    if op == "norm":
        H = _log(rng, 64, 8193)
        if rng.random() < 0.7:
            H = max(8, H // 8 * 8)
        M = _log(rng, 1, min(16384, 16384 * 7168 // H))
        groups = rng.choice((1, 1, 2, 5))
        return dict(op="norm", M=(M + groups - 1) // groups * groups, H=H, groups=groups,
                    kind=rng.choice(("rms", "layer")), dtype=rng.choice(("bf16", "bf16", "f32")),
                    post=rng.random() < 0.6, train=train)
    if op in ("linear", "experts"):
        N, K = 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 1024)
        cap = 16384 * 7168 * 2048 // (N * K)
        if op == "linear":
            M = _log(rng, 1, min(16384, cap))
            if not train and rng.random() < 0.4:
                M = rng.randint(1, 32)
            return dict(op="linear", M=M, N=N, K=K, act=rng.choice(("none", "silu", "gelu", "gelu_erf")),
                        experts=0, train=train)
        N, K = min(N, 2048), min(K, 2048)
        return dict(op="linear", M=_log(rng, 8, 16384), N=N, K=K, act=rng.choice(("none", "none", "silu")),
                    experts=rng.choice((2, 8, 24, 64)), train=train)
    H = 8 * _log(rng, 16, 896)
    k = rng.choice((1, 2, 4, 6, 8))
    E = rng.choice((8, 16, 60, 64, 128, 256))
    return dict(op="moe", T=_log(rng, 1, min(32768, 8192 * 8 * 7168 // (k * H))), k=k, E=E, H=H,
                drop=rng.choice((0.0, 0.0, 0.05, 0.5)), train=train)


# ---- inputs --------------------------------------------------------------------------------

class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, scale=1.0, shift=0.0, dtype=BF16):
        t = torch.randn(shape, generator=self.g, device="cuda", dtype=F32)
        return (t * scale + shift).to(dtype)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=F32)


def _norm_inputs(c, d):
    M, H, G = c["M"], c["H"], c["groups"]
    xt = BF16 if c["dtype"] == "bf16" else F32
    # a residual stream has a few channels far larger than the rest
    big = torch.where(d.uniform(H) < 0.004, 20.0, 1.0)
    s = dict(x=(d.normal(M, H, dtype=F32) * big).to(xt), y=d.normal(M, H, scale=0.7, shift=0.05),
             gate=d.normal(G, H, scale=0.3, shift=0.5, dtype=xt),
             w_pre=d.normal(G, H, scale=0.2, shift=1.0, dtype=xt),
             b_pre=d.normal(G, H, scale=0.1, dtype=xt) if c["kind"] == "layer" or G > 1 else None,
             w_post=d.normal(H, scale=0.2, shift=1.0, dtype=xt) if c["post"] else None,
             post=c["post"], res_scale=0.875 if c["post"] else 1.0, kind=c["kind"])
    if c["train"]:
        s.update(dx_out=d.normal(M, H, scale=0.1, dtype=xt), dh=d.normal(M, H, scale=0.1))
    return s


def _linear_inputs(c, d):
    M, N, K, E = c["M"], c["N"], c["K"], c["experts"]
    lead = (E,) if E else ()
    s = dict(x=d.normal(M, K), w=d.normal(*lead, N, K, scale=K ** -0.5), bias=d.normal(*lead, N, scale=0.3),
             residual=None if E else d.normal(M, N), act=c["act"], offsets=None)
    if E:
        # rows per expert: every row picks an expert, some experts favoured, one never chosen
        p = torch.exp(0.3 * torch.randn(E, generator=d.g, device="cuda"))
        p[E // 2] = 0.0
        pick = torch.multinomial(p, M, replacement=True, generator=d.g)
        counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, pick, torch.ones_like(pick))
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
    if c["train"]:
        s["dy"] = d.normal(M, N, scale=0.1)
    return s


def _moe_inputs(c, d):
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    logits = torch.randn((T, E), generator=d.g, device="cuda") + 0.5 * torch.randn(E, generator=d.g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    ids = torch.where(d.uniform(T, k) < c["drop"], -1, ids).to(torch.int32)
    s = dict(x=d.normal(T, H), ids=ids, weights=torch.softmax(top, 1), y=d.normal(T * k, H), E=E)
    if c["train"]:
        s.update(dout=d.normal(T, H, scale=0.1), dxs=d.normal(T * k, H, scale=0.1))
    return s


def prepare(case, seed):
    d = _Draws(seed)
    s = {"norm": _norm_inputs, "linear": _linear_inputs, "moe": _moe_inputs}[case["op"]](case, d)
    s.update(op=case["op"], train=case["train"])
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "moe": _own_moe}[state["op"]](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "moe": _plain_moe}[state["op"]](state)


def _own_norm(s):
    import glu_activation_microscaling_amd as glu
    p = dict(gate=s["gate"], w_pre=s["w_pre"], b_pre=s["b_pre"], w_post=s["w_post"], post=s["post"],
             res_scale=s["res_scale"], kind=s["kind"], eps=EPS)
    x_out, h, stats = glu.glu_block_norm(s["x"], s["y"], **p)
    if not s["train"]:
        return dict(x_out=x_out, h=h)
    dx, dy, dgate, dw_post, dw_pre, db_pre = glu.glu_block_norm_bwd(s["x"], s["y"], stats, s["dx_out"], s["dh"], **p)
    r = dict(x_out=x_out, h=h, dx=dx, dy=dy, dgate=dgate, dw_pre=dw_pre)
    if s["b_pre"] is not None:
        r["db_pre"] = db_pre
    if s["w_post"] is not None:
        r["dw_post"] = dw_post
    return r


def _own_linear(s):
    import glu_activation_microscaling_amd as glu
    if not s["train"]:
        return dict(y=glu.glu_linear(s["x"], s["w"], s["bias"], s["residual"], act=s["act"], offsets=s["offsets"]))
    pre = None
    if s["act"] == "none":
        y = glu.glu_linear(s["x"], s["w"], s["bias"], s["residual"], offsets=s["offsets"])
    else:
        y, pre = glu.glu_linear(s["x"], s["w"], s["bias"], s["residual"], act=s["act"], offsets=s["offsets"],
                                save_pre=True)
    dx, dw, db = glu.glu_linear_bwd(s["dy"], s["x"], s["w"], pre=pre, act=s["act"], offsets=s["offsets"], bias=True)
    return dict(y=y, dx=dx, dw=dw, db=db)


def _own_moe(s):
    import glu_activation_microscaling_amd as glu
    rows, offsets = glu.glu_moe_sort(s["ids"], s["E"])
    r = dict(rows=rows, offsets=offsets, xs=glu.glu_moe_permute(s["x"], rows, offsets),
             out=glu.glu_moe_combine(s["y"], rows, s["weights"]))
    if s["train"]:
        r["dy"], r["dweights"] = glu.glu_moe_combine_bwd(s["dout"], s["y"], rows, s["weights"], offsets)
        r["dx"] = glu.glu_moe_combine(s["dxs"], rows)
    return r


def _spread(p, M):
    """[G, H] parameters, one row per group of M / G consecutive rows -> FP32, one per row."""
    p = p.float()
    return p if p.shape[0] == 1 else p.repeat_interleave(M // p.shape[0], 0)


def _normed(v, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rstd = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * rstd, rstd


def _norm_grad(dn, n, rstd, kind):
    g = dn - n * (dn * n).mean(1, keepdim=True)
    if kind == "layer":
        g = g - dn.mean(1, keepdim=True)
    return g * rstd


def _plain_norm(s):
    x, M, kind = s["x"].float(), s["x"].shape[0], s["kind"]
    gate, w_pre = _spread(s["gate"], M), _spread(s["w_pre"], M)
    ny, ry = _normed(s["y"].float(), kind) if s["post"] else (s["y"].float(), None)
    z = ny * s["w_post"].float() if s["post"] else ny
    xo = s["res_scale"] * x + gate * z
    nx, rx = _normed(xo, kind)
    h = nx * w_pre
    if s["b_pre"] is not None:
        h = h + _spread(s["b_pre"], M)
    r = dict(x_out=xo.to(s["x"].dtype), h=h.to(BF16))
    if not s["train"]:
        return r
    dh, pt = s["dh"].float(), s["gate"].dtype

    def groups(t, G):
        return t.reshape(G, M // G, -1).sum(1)

    dxo = s["dx_out"].float() + _norm_grad(dh * w_pre, nx, rx, kind)
    dz = gate * dxo
    r.update(dx=(s["res_scale"] * dxo).to(s["x"].dtype),
             dgate=groups(dxo * z, s["gate"].shape[0]).to(pt), dw_pre=groups(dh * nx, s["w_pre"].shape[0]).to(pt))
    if s["b_pre"] is not None:
        r["db_pre"] = groups(dh, s["b_pre"].shape[0]).to(pt)
    if s["post"]:
        r["dw_post"] = (dz * ny).sum(0).to(pt)
        dz = _norm_grad(dz * s["w_post"].float(), ny, ry, kind)
    r["dy"] = dz.to(BF16)
    return r


def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    if act == "gelu_erf":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    return v


def _act_grad(v, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-v))
        return p * (1.0 + v * (1.0 - p))
    if act == "gelu":
        t = torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 0.134145 * v * v)
    if act == "gelu_erf":
        return 0.5 * (1.0 + torch.erf(v * 0.7071067811865476)) + 0.3989422804014327 * v * torch.exp(-0.5 * v * v)
    return torch.ones_like(v)


def _plain_linear(s):
    x, w, bias = s["x"].float(), s["w"].float(), s["bias"].float()
    off, M = s["offsets"], s["x"].shape[0]
    if off is None:
        def rows_times(t, m):
            return t @ m

        def rows_rows(a, b):
            return a.t() @ b

        pre = rows_times(x, w.t()) + bias
    else:
        # groups padded to the largest and multiplied as a batch
        slot = off[:-1, None].long() + torch.arange(s["most"], device=x.device)
        real = (slot < off[1:, None]).unsqueeze(2)
        slot = slot.clamp(max=M - 1)
        row = torch.arange(M, device=x.device)
        seg = torch.searchsorted(off[1:].long(), row, right=True)
        at = row - off[seg]

        def rows_times(t, m):
            return torch.bmm(t[slot] * real, m)[seg, at]

        def rows_rows(a, b):
            return torch.bmm((a[slot] * real).transpose(1, 2), b[slot] * real)

        pre = rows_times(x, w.transpose(1, 2)) + bias[seg]
    y = _act(pre, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    r = dict(y=y.to(BF16))
    if s["train"]:
        dpre = s["dy"].float() * _act_grad(pre, s["act"])
        r.update(dx=rows_times(dpre, w).to(BF16), dw=rows_rows(dpre, x).to(BF16),
                 db=(dpre.sum(0) if off is None else (dpre[slot] * real).sum(1)).to(BF16))
    return r


def _plain_moe(s):
    x, ids, E = s["x"], s["ids"], s["E"]
    T, k = ids.shape
    live = (ids >= 0) & (ids < E)
    key = torch.where(live, ids, E).reshape(-1).long()
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=x.device)
    rows = torch.where(live, place.reshape(T, k), -1).to(torch.int32)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)]).to(torch.int32)
    filled = (torch.arange(T * k, device=x.device) < offsets[E]).unsqueeze(1)
    at, keep = rows.clamp(min=0).long(), live.float()

    def gather(t):
        return t[at].float()

    wk = s["weights"] * keep
    r = dict(rows=rows, offsets=offsets, xs=x[order // k] * filled,
             out=(gather(s["y"]) * wk.unsqueeze(2)).sum(1).to(BF16))
    if s["train"]:
        dout = s["dout"].float()
        r["dy"] = (dout[order // k] * wk.reshape(-1)[order].unsqueeze(1) * filled).to(BF16)
        r["dweights"] = (gather(s["y"]) * dout.unsqueeze(1)).sum(2) * keep
        r["dx"] = (gather(s["dxs"]) * keep.unsqueeze(2)).sum(1).to(BF16)
    return r


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "norm":
        M, H, G, e = c["M"], c["H"], c["groups"], 2 if c["dtype"] == "bf16" else 4
        params = (2 + (c["kind"] == "layer" or G > 1)) * G * H * e + (H * e if c["post"] else 0)
        b, f = M * H * (e + 2 + e + 2) + params, 20 * M * H
        if c["train"]:  # x, y, dx_out, dh in; dx, dy and the parameters' gradients out
            b += M * H * (e + 2 + e + 2 + e + 2) + 2 * params
            f += 40 * M * H
        return {"bytes": b, "flops": f}
    if c["op"] == "linear":
        M, N, K, E = c["M"], c["N"], c["K"], max(1, c["experts"])
        res = 0 if c["experts"] else 2 * M * N
        b, f = 2 * (M * K + min(E, M) * N * K + M * N) + res, 2 * M * N * K
        if c["train"]:  # dy, x, w in; dx, dw out
            b += 2 * (M * N + 2 * M * K + 2 * min(E, M) * N * K) + (0 if c["act"] == "none" else 4 * M * N)
            f *= 3
        return {"bytes": b, "flops": f}
    T, k, H = c["T"], c["k"], c["H"]
    R = int(T * k * (1.0 - c["drop"]))
    b = 8 * T * k + 4 * c["E"] + 2 * T * H + 2 * T * k * H + 2 * R * H + 2 * T * H
    f = 2 * R * H
    if c["train"]:  # dout, y in; dy (every row), dweights out; then dxs in, dx out
        b += 2 * T * H + 2 * R * H + 2 * T * k * H + 8 * T * k + 2 * R * H + 2 * T * H
        f += 4 * R * H
    return {"bytes": b, "flops": f}


# ---- the definitions in 64 bits ------------------------------------------------------------
# Gradients here come from differentiating the forward definition, not from formulas.

def _exact_norm(s):
    D = torch.float64
    M = s["x"].shape[0]
    names = [n for n in ("x", "y", "gate", "w_pre", "b_pre", "w_post") if s[n] is not None]
    v = {n: s[n].to(D).requires_grad_(s["train"]) for n in names}

    def norm(t):
        var = t.var(1, unbiased=False, keepdim=True) if s["kind"] == "layer" else t.square().mean(1, keepdim=True)
        return (t - t.mean(1, keepdim=True) if s["kind"] == "layer" else t) / (var + EPS).sqrt()

    def rows(p):
        return p.unsqueeze(1).expand(p.shape[0], M // p.shape[0], p.shape[1]).reshape(M, -1)

    z = norm(v["y"]) * v["w_post"] if s["post"] else v["y"]
    xo = v["x"] * s["res_scale"] + rows(v["gate"]) * z
    h = norm(xo) * rows(v["w_pre"])
    if "b_pre" in v:
        h = h + rows(v["b_pre"])
    r = dict(x_out=xo.detach(), h=h.detach())
    if s["train"]:
        gs = torch.autograd.grad([xo, h], [v[n] for n in names], [s["dx_out"].to(D), s["dh"].to(D)])
        r.update({"d" + n: g for n, g in zip(names, gs)})
    return r


def _exact_linear(s):
    D, F = torch.float64, torch.nn.functional
    acts = {"none": lambda t: t, "silu": F.silu, "gelu": lambda t: F.gelu(t, approximate="tanh"), "gelu_erf": F.gelu}
    off = [0, s["x"].shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    y = torch.zeros(s["x"].shape[0], s["w"].shape[-2], dtype=D, device="cuda")
    dx = torch.zeros(s["x"].shape, dtype=D, device="cuda")
    dw, db = [], []
    for e in range(len(off) - 1):
        a, b = off[e], off[e + 1]
        w, bias = (s["w"], s["bias"]) if s["offsets"] is None else (s["w"][e], s["bias"][e])
        x, w, bias = s["x"][a:b].to(D), w.to(D), bias.to(D)
        pre = (x @ w.t() + bias).requires_grad_(s["train"])
        out = acts[s["act"]](pre)
        y[a:b] = out.detach()
        if s["residual"] is not None:
            y[a:b] += s["residual"][a:b].to(D)
        if s["train"]:
            dy = s["dy"][a:b].to(D)
            dp = torch.autograd.grad(out, pre, dy)[0] if b > a and s["act"] != "none" else dy
            dx[a:b] = dp @ w
            dw.append(dp.t() @ x)
            db.append(dp.sum(0))
    r = dict(y=y)
    if s["train"]:
        one = s["offsets"] is None
        r.update(dx=dx, dw=dw[0] if one else torch.stack(dw), db=db[0] if one else torch.stack(db))
    return r


def _exact_moe(s):
    D = torch.float64
    ids = s["ids"].cpu()
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    queue = [[] for _ in range(s["E"])]
    for i, e in enumerate(flat):
        if 0 <= e < s["E"]:
            queue[e].append(i)
    src = [i for q in queue for i in q]
    ends = [0]
    for q in queue:
        ends.append(ends[-1] + len(q))
    rows = torch.full((T * k,), -1, dtype=torch.int32)
    src = torch.tensor(src, dtype=torch.int64)
    rows[src] = torch.arange(len(src), dtype=torch.int32)
    src = src.cuda()
    n, tok = len(src), src // k
    w = s["weights"].reshape(-1).to(D)[src].unsqueeze(1)

    def back(t):  # [n, H] rows added to their tokens
        return torch.zeros(T, t.shape[1], dtype=D, device="cuda").index_add_(0, tok, t)

    xs = torch.zeros(T * k, s["x"].shape[1], dtype=D, device="cuda")
    xs[:n] = s["x"].to(D)[tok]
    y = s["y"][:n].to(D)
    r = dict(rows=rows.reshape(T, k).cuda(), offsets=torch.tensor(ends, dtype=torch.int32).cuda(), xs=xs,
             out=back(y * w))
    if s["train"]:
        g = s["dout"].to(D)[tok]
        dy = torch.zeros_like(xs)
        dy[:n] = g * w
        dweights = torch.zeros(T * k, dtype=D, device="cuda")
        dweights[src] = (g * y).sum(1)
        r.update(dy=dy, dweights=dweights.reshape(T, k), dx=back(s["dxs"][:n].to(D)))
    return r


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "moe": _exact_moe}[case["op"]](s)

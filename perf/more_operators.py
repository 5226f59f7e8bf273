"""Cases that measure the gated projection, its 8-bit checkpoints, and products in 8-bit floating
point.

Three groups of operators, each in the forms a feed-forward block uses:

  gated    h = act(x Wg^T + bg) * (x Wu^T + bu) in one call; with "train" also dx, dW and db,
           gate and up kept in between as BF16 ("save": "bf16") or as E4M3 codes with a
           power-of-two scale for each 32 of a row ("save": "mxfp8").  "experts" > 0: row groups
           given by offsets, one W and b per group.
  ckpt     h = act(gate) * up with gate and up kept as such codes, and the backward pass
           from the codes: the gradients of gate and up, and h formed again.
  fp8      serving: the GLU of gate and up quantized to E4M3 with a scale for each 128 of a row,
           times weights in E4M3 with a scale for each 128 x 128.  "train": y = x W^T and both
           gradients from operands quantized on the way, all three products in 8 bits.

`own` selects between the plain form (elementary torch operations, FP32 products) and the
library's entry points.  A case is a dict of plain values; `prepare` makes the tensors of a case
from a seed, `run` is one pass, `exact` the same results in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("swiglu", "geglu", "geglu_erf", "relu2")


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # gate and up projections of one new token: one pass over both matrices
        dict(name="gated-token", op="gated", M=1, N=16384, K=2048, act="geglu", layout="paired", bias=False,
             experts=0, save="none"),
        # the same projections of a prefill
        dict(name="gated-prefill", op="gated", M=968, N=16384, K=2048, act="geglu", layout="paired", bias=False,
             experts=0, save="none"),
        # a training step at the library's large activation shape
        dict(name="gated-train", op="gated", M=16384, N=7168, K=2048, act="swiglu", layout="split", bias=False,
             experts=0, save="bf16"),
        # a small ragged training step with biases and 8-bit checkpoints: no extent is a multiple of a tile
        dict(name="gated-train-odd", op="gated", M=1021, N=1000, K=2056, act="geglu_erf", layout="paired", bias=True,
             experts=0, save="mxfp8"),
        # a training step of 16 experts with 8-bit checkpoints
        dict(name="gated-experts-train", op="gated", M=16384, N=2048, K=2048, act="swiglu", layout="split",
             bias=False, experts=16, save="mxfp8"),
        # the smallest activation of the library's own benchmark: launch latency
        dict(name="ckpt-small", op="ckpt", M=128, N=128, act="swiglu"),
        # a training step's activation
        dict(name="ckpt-train", op="ckpt", M=16384, N=7168, act="swiglu"),
        # a ragged activation: rows end inside a block of 32
        dict(name="ckpt-odd", op="ckpt", M=1021, N=1000, act="geglu_erf"),
        # the down projection of one new token: one pass over the 8-bit weights
        dict(name="fp8-token", op="fp8", M=1, N=2048, K=16384, act="geglu", experts=0, train=False),
        # the same projection of a prefill
        dict(name="fp8-prefill", op="fp8", M=968, N=2048, K=16384, act="geglu", experts=0, train=False),
        # the down projections of 16 experts for a batch of routed rows
        dict(name="fp8-experts", op="fp8", M=8192, N=4096, K=2048, act="swiglu", experts=16, train=False),
        # a large training step in 8 bits
        dict(name="fp8-train", op="fp8", M=16384, N=7168, K=2048, act="none", experts=0, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "gated", "ckpt", "fp8", "fp8"))
    if op == "ckpt":
        N = 8 * _log(rng, 16, 2048)
        return dict(op="ckpt", M=_log(rng, 1, min(16384, 16384 * 7168 // N)), N=N, act=rng.choice(ACTS))
    N, K = 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 1024)
    experts = rng.choice((0, 0, 2, 8, 24, 64))
    if experts:
        N, K = min(N, 2048), min(K, 2048)
    M = _log(rng, 1, min(16384, 16384 * 7168 * 2048 // (N * K)))
    if op == "gated":
        save = rng.choice(("none", "none", "bf16", "mxfp8"))
        if save == "none" and not experts and rng.random() < 0.4:
            M = rng.randint(1, 32)
        return dict(op="gated", M=M, N=N, K=K, act=rng.choice(ACTS), layout=rng.choice(("split", "paired")),
                    bias=rng.random() < 0.4, experts=experts, save=save)
    K = 16 * (K // 16)
    train = not experts and rng.random() < 0.5
    if not train and not experts and rng.random() < 0.4:
        M = rng.randint(1, 32)
    return dict(op="fp8", M=M, N=N, K=K, act="none" if train else rng.choice(ACTS), experts=experts, train=train)


# ---- inputs --------------------------------------------------------------------------------

class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, scale=1.0, dtype=BF16):
        t = torch.randn(shape, generator=self.g, device="cuda", dtype=F32)
        return (t * scale).to(dtype)

    def wide(self, M, N):
        """Activations as they come: a few channels far larger than the rest."""
        big = torch.where(torch.rand(N, generator=self.g, device="cuda") < 0.004, 20.0, 1.0)
        return (torch.randn((M, N), generator=self.g, device="cuda") * big).to(BF16)

    def groups(self, M, E):
        """Rows per expert: every row picks one, some favoured, one never chosen."""
        p = torch.exp(0.3 * torch.randn(E, generator=self.g, device="cuda"))
        p[E // 2] = 0.0
        pick = torch.multinomial(p, M, replacement=True, generator=self.g)
        counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, pick, torch.ones_like(pick))
        return dict(offsets=torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), most=int(counts.max()))


def prepare(case, seed):
    c, d = case, _Draws(seed)
    s = dict(case, offsets=None)
    M, N = c["M"], c["N"]
    if c["op"] == "ckpt":
        s.update(gate=d.wide(M, N), up=d.wide(M, N), dh=d.normal(M, N, scale=0.1))
        return s
    K, E = c["K"], c["experts"]
    lead = (E,) if E else ()
    if E:
        s.update(d.groups(M, E))
    if c["op"] == "gated":
        s.update(x=d.normal(M, K), w=d.normal(*lead, 2 * N, K, scale=K ** -0.5),
                 b=d.normal(*lead, 2 * N, scale=0.3) if c["bias"] else None)
        if c["save"] != "none":
            s["dh"] = d.normal(M, N, scale=0.1)
        return s
    w = d.normal(*lead, N, K, scale=K ** -0.5)
    if c["train"]:
        s.update(x=d.wide(M, K), w=w, dy=d.normal(M, N, scale=0.1))
        return s
    # serving keeps the weights in 8 bits: codes and the scale of each 128 x 128 block
    q, sc = _fp8(w.float(), 128, 128)
    s.update(gate=d.normal(M, K), up=d.wide(M, K), wq=q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(),
             ws=sc.contiguous())
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(state):
    if own:
        return {"gated": _own_gated, "ckpt": _own_ckpt, "fp8": _own_fp8}[state["op"]](state)
    return {"gated": _plain_gated, "ckpt": _plain_ckpt, "fp8": _plain_fp8}[state["op"]](state)


def _own_gated(s):
    import glu_activation_microscaling_amd as glu
    p = dict(act=s["act"], w_layout=s["layout"], offsets=s["offsets"])
    if s["save"] == "none":
        return dict(h=glu.glu_gated_linear(s["x"], s["w"], s["b"], **p))
    h, pre, scales = glu.glu_gated_linear(s["x"], s["w"], s["b"], save=s["save"], **p)
    dx, dw, db, _ = glu.glu_gated_linear_bwd(s["dh"], s["x"], s["w"], pre, scales, bias=s["bias"], **p)
    r = dict(h=h, dx=dx, dw=dw)
    if s["bias"]:
        r["db"] = db
    return r


def _own_ckpt(s):
    import glu_activation_microscaling_amd as glu
    h, q, scales = glu.glu_fwd_ckpt(s["gate"], s["up"], act=s["act"])
    d, again = glu.glu_bwd_ckpt(q, scales, s["dh"], act=s["act"], need_h=True)
    return dict(h=h, d=d, again=again)


def _own_fp8(s):
    import glu_activation_microscaling_amd as glu
    if not s["train"]:
        q, _, sc, _ = glu.glu_fwd_fp8(s["gate"], s["up"], act=s["act"])
        return dict(y=glu.glu_linear_fp8(q, sc, s["wq"], s["ws"], offsets=s["offsets"]))
    xr, xc, sxr, sxc = glu.glu_quant_fp8(s["x"], rowwise=True, colwise=True)
    wq, ws, wt, wts = glu.glu_quant_fp8_weight(s["w"], transpose=True)
    y = glu.glu_linear_fp8(xr, sxr, wq, ws)
    dr, dc, sdr, sdc = glu.glu_quant_fp8(s["dy"], rowwise=True, colwise=True)
    dx = glu.glu_linear_fp8(dr, sdr, wt, wts)
    dw = glu.glu_linear_fp8(dc, sdc, xc, sxc, w_scales="row")
    return dict(y=y, dx=dx, dw=dw)


def _act(g, act):
    if act == "swiglu":
        return g / (1.0 + torch.exp(-g))
    if act == "geglu":
        return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))
    if act == "geglu_erf":
        return 0.5 * g * (1.0 + torch.erf(g * 0.7071067811865476))
    return torch.clamp(g, min=0.0) ** 2


def _act_grad(g, act):
    if act == "swiglu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    if act == "geglu":
        t = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 0.134145 * g * g)
    if act == "geglu_erf":
        return 0.5 * (1.0 + torch.erf(g * 0.7071067811865476)) + 0.3989422804014327 * g * torch.exp(-0.5 * g * g)
    return 2.0 * torch.clamp(g, min=0.0)


def _blocks(v, rows, cols):
    """[..., M, N] cut into blocks of rows x cols, the last ones filled up with zeros."""
    M, N = v.shape[-2:]
    v = torch.nn.functional.pad(v, (0, -N % cols, 0, -M % rows))
    return v.reshape(*v.shape[:-2], v.shape[-2] // rows, rows, v.shape[-1] // cols, cols)


def _back(b, M, N):
    *lead, i, r, j, c = b.shape
    return b.reshape(*lead, i * r, j * c)[..., :M, :N]


def _e4m3(v):
    return v.to(F32).to(torch.float8_e4m3fn).to(F32)


def _fp8(v, rows, cols):
    """E4M3 values of v and the scale of each block of rows x cols: the block's largest magnitude
    (2^-100 at least) stands for 448.  Which code is nearest is decided in 64 bits."""
    b = _blocks(v, rows, cols)
    top = b.abs().amax((-3, -1), keepdim=True).clamp(min=2.0 ** -100)
    q = _e4m3((b.double() * 448.0) / top.double())
    return _back(q, *v.shape[-2:]), (top / 448.0)[..., 0, :, 0]


def _fp8_values(v, rows, cols):
    M, N = v.shape[-2:]
    q, s = _fp8(v, rows, cols)
    return q * s.repeat_interleave(rows, -2)[..., :M, :].repeat_interleave(cols, -1)[..., :N]


def _mx_values(v):
    """What E4M3 codes with a power-of-two scale for each 32 of a row of BF16 values stand for."""
    b = _blocks(v.to(BF16).float(), 1, 32)
    m, e = torch.frexp(b.abs().amax((-3, -1), keepdim=True) / 448.0)
    e = torch.where(m > 0.5, e, e - 1).clamp(min=-127)       # the least with 448 2^e >= the largest
    return _back(torch.ldexp(_e4m3(torch.ldexp(b, -e)), e), *v.shape[-2:])


class _Groups:
    """Products of rows with their group's matrix: groups padded to the largest, as a batch."""

    def __init__(self, s, M):
        off = s["offsets"]
        slot = off[:-1, None].long() + torch.arange(s["most"], device=off.device)
        self.real = (slot < off[1:, None]).unsqueeze(2)
        self.slot = slot.clamp(max=M - 1)
        row = torch.arange(M, device=off.device)
        self.seg = torch.searchsorted(off[1:].long(), row, right=True)
        self.at = row - off[self.seg]

    def take(self, t):
        return t[self.slot] * self.real

    def times(self, t, m):
        return torch.bmm(self.take(t), m)[self.seg, self.at]


def _joined(a, b, layout):
    """[M, 2N] in the order of W's rows."""
    return torch.cat([a, b], 1) if layout == "split" else torch.stack([a, b], 2).flatten(1)


def _plain_gated(s):
    x, w, act, layout, N = s["x"].float(), s["w"].float(), s["act"], s["layout"], s["N"]
    grouped = s["offsets"] is not None
    G = _Groups(s, x.shape[0]) if grouped else None
    pre = G.times(x, w.transpose(1, 2)) if grouped else x @ w.t()
    if s["b"] is not None:
        b = s["b"].float()
        pre = pre + (b[G.seg] if grouped else b)
    if layout == "split":
        g, u = pre[:, :N], pre[:, N:]
    else:
        g, u = pre[:, 0::2], pre[:, 1::2]
    r = dict(h=(_act(g, act) * u).to(BF16))
    if s["save"] == "none":
        return r
    if s["save"] == "mxfp8":
        g, u = _mx_values(g), _mx_values(u)
    dh = s["dh"].float()
    dp = _joined(dh * u * _act_grad(g, act), dh * _act(g, act), layout)
    if grouped:
        r.update(dx=G.times(dp, w).to(BF16), dw=torch.bmm(G.take(dp).transpose(1, 2), G.take(x)).to(BF16))
        if s["bias"]:
            r["db"] = G.take(dp).sum(1).to(BF16)
    else:
        r.update(dx=(dp @ w).to(BF16), dw=(dp.t() @ x).to(BF16))
        if s["bias"]:
            r["db"] = dp.sum(0).to(BF16)
    return r


def _plain_ckpt(s):
    g, u, dh, act = s["gate"].float(), s["up"].float(), s["dh"].float(), s["act"]
    r = dict(h=(_act(g, act) * u).to(BF16))
    g, u = _mx_values(g), _mx_values(u)
    a = _act(g, act)
    r["d"] = torch.cat([(dh * u * _act_grad(g, act)).to(BF16), (dh * a).to(BF16)], 1)
    r["again"] = (a * u).to(BF16)
    return r


def _plain_fp8(s):
    if not s["train"]:
        h = (_act(s["gate"].float(), s["act"]) * s["up"].float()).to(BF16)
        x, N, K = _fp8_values(h.float(), 1, 128), s["N"], s["K"]
        w = s["wq"].view(torch.float8_e4m3fn).float()
        w = w * s["ws"].repeat_interleave(128, -2)[..., :N, :].repeat_interleave(128, -1)[..., :K]
        y = x @ w.t() if s["offsets"] is None else _Groups(s, x.shape[0]).times(x, w.transpose(1, 2))
        return dict(y=y.to(BF16))
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    wv = _fp8_values(w, 128, 128)
    return dict(y=(_fp8_values(x, 1, 128) @ wv.t()).to(BF16), dx=(_fp8_values(dy, 1, 128) @ wv).to(BF16),
                dw=(_fp8_values(dy, 128, 1).t() @ _fp8_values(x, 128, 1)).to(BF16))


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    c = case
    M, N = c["M"], c["N"]
    if c["op"] == "ckpt":
        # gate and up in, h and codes out; codes and dh in, both gradients and h out
        kept = 2 * M * (N + (N + 31) // 32)
        return {"bytes": 6 * M * N + 8 * M * N + 2 * kept, "flops": 40 * M * N}
    K, E = c["K"], c["experts"]
    used = min(max(1, E - 1), M)                    # groups that have rows; one never has
    if c["op"] == "gated":
        b, f = 2 * (M * K + used * 2 * N * K + M * N), 4 * M * N * K
        if c["save"] != "none":                     # dh in; dx and dW (every group's) out
            b += 2 * (M * N + M * K + max(1, E) * 2 * N * K)
            f *= 3
        return {"bytes": b, "flops": f}
    if not c["train"]:                              # gate, up, 8-bit weights in; y out
        return {"bytes": 4 * M * K + used * N * K + 2 * M * N, "flops": 2 * M * N * K}
    return {"bytes": 2 * (2 * M * K + 2 * N * K + 2 * M * N), "flops": 6 * M * N * K}


# ---- the definitions in 64 bits ------------------------------------------------------------
# Gradients here come from differentiating the forward definition, codes from rounding to the
# formats' grids by arithmetic.

D = torch.float64


def _glu64(g, u, act):
    F = torch.nn.functional
    f = {"swiglu": F.silu, "geglu": lambda t: F.gelu(t, approximate="tanh"), "geglu_erf": F.gelu,
         "relu2": lambda t: F.relu(t).square()}[act]
    return f(g) * u


def _grid(y):
    """The nearest multiple of E4M3's step at |y|: 2^(e - 3), at least 2^-9; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def _by_blocks(v, rows, cols, f):
    """f(block values, block maxima) for each block of a matrix, the maxima spread over it."""
    M, N = v.shape
    m = v.abs()
    if cols > 1:
        m = torch.stack([p.amax(1) for p in m.split(cols, 1)], 1)
    if rows > 1:
        m = torch.stack([p.amax(0) for p in m.split(rows, 0)], 0)
    i, j = torch.arange(M, device=v.device) // rows, torch.arange(N, device=v.device) // cols
    return f(v, m[i][:, j])


def _fp8_64(v, rows, cols):
    def f(x, m):
        m = m.clamp(min=2.0 ** -100)
        return _grid(x * 448.0 / m) * (m / 448.0)
    return _by_blocks(v, rows, cols, f)


def _mx_64(v):
    def f(x, m):
        q = m / 448.0
        e = torch.floor(torch.log2(q.clamp(min=2.0 ** -200)))
        e = torch.where(torch.exp2(e) >= q, e, e + 1.0).clamp(min=-127.0)
        return _grid(x * torch.exp2(-e)) * torch.exp2(e)
    return _by_blocks(v.to(BF16).to(D), 1, 32, f)


def _exact_gated(s):
    M, N, split, train = s["M"], s["N"], s["layout"] == "split", s["save"] != "none"
    off = [0, M] if s["offsets"] is None else s["offsets"].tolist()
    one = s["offsets"] is None
    h = torch.zeros(M, N, dtype=D, device="cuda")
    dx = torch.zeros(s["x"].shape, dtype=D, device="cuda")
    dw, db = [], []
    for e, (i, j) in enumerate(zip(off[:-1], off[1:])):
        w = (s["w"] if one else s["w"][e]).to(D)
        x = s["x"][i:j].to(D)
        g, u = x @ (w[:N] if split else w[0::2]).t(), x @ (w[N:] if split else w[1::2]).t()
        if s["b"] is not None:
            b = (s["b"] if one else s["b"][e]).to(D)
            g, u = g + (b[:N] if split else b[0::2]), u + (b[N:] if split else b[1::2])
        h[i:j] = _glu64(g, u, s["act"])
        if train:
            if s["save"] == "mxfp8" and j > i:
                g, u = _mx_64(g), _mx_64(u)
            g, u = g.requires_grad_(True), u.requires_grad_(True)
            a, c = torch.autograd.grad(_glu64(g, u, s["act"]), [g, u], s["dh"][i:j].to(D))
            dp = torch.empty(j - i, 2 * N, dtype=D, device="cuda")
            dp[:, slice(0, N) if split else slice(0, None, 2)] = a
            dp[:, slice(N, None) if split else slice(1, None, 2)] = c
            dx[i:j] = dp @ w
            dw.append(dp.t() @ x)
            db.append(dp.sum(0))
    r = dict(h=h)
    if train:
        r.update(dx=dx, dw=dw[0] if one else torch.stack(dw))
        if s["bias"]:
            r["db"] = db[0] if one else torch.stack(db)
    return r


def _exact_ckpt(s):
    h = _glu64(s["gate"].to(D), s["up"].to(D), s["act"])
    g, u = _mx_64(s["gate"]).requires_grad_(True), _mx_64(s["up"]).requires_grad_(True)
    again = _glu64(g, u, s["act"])
    a, b = torch.autograd.grad(again, [g, u], s["dh"].to(D))
    return dict(h=h, d=torch.cat([a, b], 1), again=again.detach())


def _exact_fp8(s):
    if s["train"]:
        x, w, dy = s["x"].to(D), s["w"].to(D), s["dy"].to(D)
        w = _fp8_64(w, 128, 128)
        return dict(y=_fp8_64(x, 1, 128) @ w.t(), dx=_fp8_64(dy, 1, 128) @ w,
                    dw=_fp8_64(dy, 128, 1).t() @ _fp8_64(x, 128, 1))
    M, N, K = s["M"], s["N"], s["K"]
    h = _glu64(s["gate"].to(D), s["up"].to(D), s["act"]).to(BF16).to(D)     # the quantizer sees BF16
    x = _fp8_64(h, 1, 128)
    off = [0, M] if s["offsets"] is None else s["offsets"].tolist()
    y = torch.zeros(M, N, dtype=D, device="cuda")
    i, j = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        q, sc = (s["wq"], s["ws"]) if s["offsets"] is None else (s["wq"][e], s["ws"][e])
        w = q.view(torch.float8_e4m3fn).to(D) * sc.to(D)[i][:, j]
        y[a:b] = x[a:b] @ w.t()
    return dict(y=y)


def exact(case, seed):
    s = prepare(case, seed)
    return {"gated": _exact_gated, "ckpt": _exact_ckpt, "fp8": _exact_fp8}[case["op"]](s)

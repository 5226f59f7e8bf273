"""Binding of the gated projections and of the GLU's 8-bit checkpoints.

Argument marshalling only, as for the other entry points (C names and formulas in
include/glu_mx.h); every function is also a name of the package:
  glu_gated_linear(x, w, bias, act=, w_layout=, offsets=, save=)  -> h, or (h, pre, extra)
  glu_gated_linear_bwd(dh, x, w, pre, extra, ...)                -> (dx, dw, db, h)
  glu_fwd_ckpt(gate, up, act=, layout=)                           -> (h, q, s)
  glu_bwd_ckpt(q, s, dh, act=, layout=)                           -> (d, h)
What is disabled comes back zero-sized (fixed arity).  Scratch memory is a torch allocation of
the call, on the current stream.
"""
import torch

from . import ACT, LAYOUT, W_LAYOUT, _operands
from .ffn import _BF16, _I32, _allocator, _launch, _like, _matrix, _ptr, _same_device, _size

SAVE = {"none": 0, "bf16": 1, "mxfp8": 2}
_U8 = torch.uint8


def _choice(value, table, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return table[value]


def _glu_operands(gate, up, layout):
    """(M, N, row stride) of the GLU's operands."""
    ld = _matrix(gate, "gate", _BF16)
    M, C = gate.shape
    if layout == "paired":
        if up is not None or C % 2:
            _operands(gate, up, layout)   # says what is wrong
        return M, C // 2, ld
    if up is None or _matrix(up, "up", _BF16) != ld or up.shape != gate.shape:
        _operands(gate, up, layout)
        raise ValueError("gate and up must share a row stride")
    return M, C, ld


def _gated_setup(x, w, bias, offsets, act, w_layout):
    a, layout = _choice(act, ACT, "act"), _choice(w_layout, W_LAYOUT, "w_layout")
    if w.dim() not in (2, 3) or w.shape[-2] % 2:
        raise ValueError("w must be [2N, K], or [groups, 2N, K] with offsets")
    if (w.dim() == 3) != (offsets is not None):
        raise ValueError("offsets go with w [groups, 2N, K], and only with it")
    N, K = w.shape[-2] // 2, w.shape[-1]
    groups = w.shape[0] if w.dim() == 3 else 1
    _like(w, "w", _BF16, w.shape)
    ld_x = _matrix(x, "x", _BF16, None, K)
    if bias is not None:
        _like(bias, "bias", _BF16, w.shape[:-1])
    if offsets is not None:
        _like(offsets, "offsets", _I32, (groups + 1,))
    return a, layout, x.shape[0], N, K, groups, ld_x


def _scale_columns(N):
    return 2 * ((N + 31) // 32)


def glu_gated_linear(x, w, bias=None, *, act="swiglu", w_layout="split", offsets=None, save="none", out=None):
    """h = act(x Wg^T + bg) * (x Wu^T + bu), [M, N].  w [2N, K] and bias [2N] hold gates above ups
    (w_layout "split") or in turn ("paired"); with int32 offsets [groups + 1], w is [groups, 2N, K],
    rows offsets[e] .. offsets[e + 1] - 1 of x go through w[e] and bias[e], and rows of no group give
    zeros.  save="bf16" or "mxfp8" returns (h, pre, extra) with what glu_gated_linear_bwd takes,
    [gate | up]: BF16 pre [M, 2N] with four more bits of each value in extra [M, N], or E4M3 codes
    [M, 2N] with E8M0 scales [M, 2 ceil(N/32)]."""
    a, layout, M, N, K, groups, ld_x = _gated_setup(x, w, bias, offsets, act, w_layout)
    keep = _choice(save, SAVE, "save")
    _same_device(x, w, bias, offsets, out)
    new = _allocator(x)
    if out is None:
        h, ld_h = new((M, N), _BF16), N
    else:
        h, ld_h = out, _matrix(out, "out", _BF16, M, N)
    pre = extra = None
    if keep:
        pre = new((M, 2 * N), _BF16 if keep == 1 else _U8)
        extra = new((M, N if keep == 1 else _scale_columns(N)), _U8)
    nbytes = _size("glu_gated_linear_work_bytes", keep, M, N, K, groups, int(offsets is not None))
    work = new((nbytes,), _U8) if nbytes > 0 else None
    _launch(x, "glu_gated_linear", a, layout, keep, M, N, K, groups, _ptr(offsets), _ptr(x), ld_x, _ptr(w), _ptr(bias),
          _ptr(h), ld_h, _ptr(pre), _ptr(extra), _ptr(work), nbytes)
    return (h, pre, extra) if keep else h


def glu_gated_linear_bwd(dh, x, w, pre, extra=None, *, act="swiglu", w_layout="split", offsets=None, bias=False,
                         need_dx=True, need_dw=True, need_h=False):
    """Gradients of glu_gated_linear from what its save kept (pre and extra; BF16 pre may come alone), taken
    at the values kept: (dx [M, K], dw like w, db [2N] or [groups, 2N] in w's order, h [M, N] formed again).
    bias=True asks for db.  What is not wanted comes back zero-sized."""
    a, layout, M, N, K, groups, ld_x = _gated_setup(x, w, None, offsets, act, w_layout)
    ld_dh = _matrix(dh, "dh", _BF16, M, N)
    keep = 2 if pre.dtype is _U8 else 1
    if extra is not None and keep == 1 and extra.numel() == 0:
        extra = None
    if extra is not None:
        _like(extra, "extra", _U8, (M, N if keep == 1 else _scale_columns(N)))
    elif keep == 2:
        raise ValueError("codes need their scales")
    _like(pre, "pre", _U8 if keep == 2 else _BF16, (M, 2 * N))
    _same_device(x, w, dh, pre, extra, offsets)
    new = _allocator(x)
    dx = new((M, K) if need_dx else (0,), _BF16)
    dw = new(w.shape if need_dw else (0,), _BF16)
    db = new(w.shape[:-1] if bias else (0,), _BF16)
    h = new((M, N) if need_h else (0,), _BF16)
    nbytes = _size("glu_gated_linear_bwd_work_bytes", M, N, K, groups, int(offsets is not None), int(bias))
    work = new((nbytes,), _U8) if nbytes > 0 else None
    _launch(x, "glu_gated_linear_bwd", a, layout, keep, M, N, K, groups, _ptr(offsets), _ptr(dh), ld_dh, _ptr(x), ld_x,
          _ptr(w), _ptr(pre), _ptr(extra), _ptr(dx) if need_dx else None, K, _ptr(dw) if need_dw else None,
          _ptr(db) if bias else None, _ptr(h) if need_h else None, N, _ptr(work), nbytes)
    return dx, dw, db, h


def glu_fwd_ckpt(gate, up=None, *, act="swiglu", layout="split", need_h=True, out=None):
    """(h [M, N], q [M, 2N], s [M, 2 ceil(N/32)]): h = act(gate) * up as glu_fwd, and the MXFP8 codes
    and scales of [gate | up] that glu_bwd_ckpt takes in place of gate and up.  need_h=False leaves h
    zero-sized."""
    a, lay = _choice(act, ACT, "act"), _choice(layout, LAYOUT, "layout")
    M, N, ld = _glu_operands(gate, up, layout)
    _same_device(gate, up, out)
    new = _allocator(gate)
    if not need_h:
        if out is not None:
            raise ValueError("out is for h (need_h=True)")
        h, ld_h = new((0,), _BF16), 0
    elif out is None:
        h, ld_h = new((M, N), _BF16), N
    else:
        h, ld_h = out, _matrix(out, "out", _BF16, M, N)
    q, s = new((M, 2 * N), _U8), new((M, _scale_columns(N)), _U8)
    _launch(gate, "glu_fwd_ckpt", a, lay, M, N, _ptr(gate), _ptr(up), ld, _ptr(h) if need_h else None, ld_h, _ptr(q), _ptr(s))
    return h, q, s


def glu_bwd_ckpt(q, s, dh, *, act="swiglu", layout="split", need_h=False, out=None):
    """(d [M, 2N], h [M, N]): the gradients of gate and up, [da | db] (layout "split") or in turn
    ("paired"), at the values that glu_fwd_ckpt's q and s stand for, and act(gate) * up of those values
    (zero-sized without need_h)."""
    a, lay = _choice(act, ACT, "act"), _choice(layout, LAYOUT, "layout")
    ld_dh = _matrix(dh, "dh", _BF16)
    M, N = dh.shape
    _like(q, "q", _U8, (M, 2 * N))
    _like(s, "s", _U8, (M, _scale_columns(N)))
    _same_device(dh, q, s, out)
    new = _allocator(dh)
    if out is None:
        d, ld_d = new((M, 2 * N), _BF16), 2 * N
    else:
        d, ld_d = out, _matrix(out, "out", _BF16, M, 2 * N)
    h = new((M, N) if need_h else (0,), _BF16)
    _launch(dh, "glu_bwd_ckpt", a, lay, M, N, _ptr(q), _ptr(s), _ptr(dh), ld_dh, _ptr(d), ld_d, _ptr(h) if need_h else None, N)
    return d, h

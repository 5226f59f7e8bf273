"""Binding of the operators around the GLU: block norms, linear products, expert routing.

Argument marshalling only, as for the GLU entry points (C names and formulas in
include/glu_mx.h); every function is also a name of the package:
  glu_block_norm(x, y=None, ...)               -> (x_out, h, stats)
  glu_block_norm_mxfp8(x, y=None, ...)         -> (x_out, q, s, stats), h quantized rowwise
  glu_block_norm_bwd(x, y, stats, dx_out, dh, ...) -> (dx, dy, dgate, dw_post, dw_pre, db_pre)
  glu_linear(x, w, bias, residual, ...)        -> y, or (y, pre) with save_pre
  glu_linear_bwd(dy, x, w, ...)                -> (dx, dw, db)
  glu_moe_sort(ids, experts)                   -> (rows, offsets)
  glu_moe_permute(x, rows, offsets)            -> xs
  glu_moe_combine(y, rows, weights, residual)  -> out
  glu_moe_combine_bwd(dout, y, rows, weights, offsets) -> (dy, dweights)
What is disabled comes back zero-sized (fixed arity).  Scratch memory is a torch allocation of
the call, on the current stream.
"""
import torch

from . import GluError, _rowmajor, lib

NORM_KIND = {"rms": 0, "layer": 1}
LINEAR_ACT = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 2, "gelu_erf": 3}
_PRE, _POST, _F32_STREAM, _F32_PARAMS, _GATE_GROUPED, _W_GROUPED, _B_GROUPED = 1, 2, 4, 8, 16, 32, 64

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


_fns = {}   # C entry points by name, looked up once


def _call(name, *args):
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    status = fn(*args)
    if status != 0:
        raise GluError(name, status)


def _size(name, *args):
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    return fn(*args)


# The current stream's handle by device index: what torch.cuda.current_stream(device).cuda_stream
# is, without the stream object in between (0.2 us instead of 2.3).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


_device = getattr(torch._C, "_cuda_getDevice", None)   # torch.cuda.current_device() without its checks


def _launch(t, name, *args):
    """_call on t's device, whichever is current, with the current stream of that device."""
    dev = t.get_device()
    if (torch.cuda.current_device() if _device is None else _device()) == dev:
        return _call(name, *args, _stream(t))
    with torch.cuda.device(dev):
        return _call(name, *args, _stream(t))


_GPU = torch.device("cuda")   # the current one


def _strided(shape, stride, dtype):
    return torch.empty_strided(shape, stride, dtype=dtype, device=_GPU)   # 1.3 us where new_empty takes 1.5


def _contiguous(shape, dtype):
    if len(shape) == 2:
        m, n = shape
        return _strided((m, n), (n or 1, 1), dtype)   # tuples alone will do
    stride = [1] * len(shape)
    for i in range(len(shape) - 1, 0, -1):
        stride[i - 1] = stride[i] * (shape[i] or 1)
    return _strided(tuple(shape), tuple(stride), dtype)


def _allocator(t):
    """new(shape, dtype): uninitialised contiguous tensors on GPU tensor t's device."""
    if _strided is None or _device is None or _device() != t.get_device():
        return lambda shape, dtype: t.new_empty(shape, dtype=dtype)
    return _contiguous


def _ptr(t):
    return None if t is None else t.data_ptr() or None   # an empty tensor's pointer is 0


def _matrix(t, name, dtype, rows=None, cols=None):
    """Row stride of a 2-D GPU tensor with unit column stride (of [rows, cols] where given).
    The stride of a single row means nothing; a whole number of vectors is passed for it.  No stride
    of a tensor without rows does: the gradient of a sum over one is expanded, and contiguous."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not dtype or not t.is_cuda or len(shape) != 2 or (stride[1] != 1 and shape[1] > 1 and shape[0] > 0):
        _rowmajor(t, name, dtype)   # says what is wrong
    M, N = shape
    if (rows is not None and M != rows) or (cols is not None and N != cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got [{M}, {N}]")
    return stride[0] if M > 1 else _one_row(N)


def _one_row(N):
    return (N + 7) // 8 * 8


def _empty(t, shape, dtype):
    """An uninitialised tensor on t's device; shaped like a contiguous t it is the quicker call."""
    if dtype is t.dtype and t.shape == shape and t.is_contiguous():
        return torch.empty_like(t)
    return t.new_empty(shape, dtype=dtype)


def _like(t, name, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous GPU tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


def _same_device(ref, *tensors):
    dev = ref.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"the operands are on different devices: {t.device} and {ref.device}")


# ---- norms -----------------------------------------------------------------------------------

def _norm_setup(x, y, gate, w_pre, b_pre, w_post, pre, post, kind):
    """(kind code, flags, M, H, groups, ld_x, ld_y) of a norm call, its parameters checked."""
    if kind not in NORM_KIND:
        raise ValueError(f"kind must be one of {sorted(NORM_KIND)}")
    if x.dtype not in (_BF16, _F32):
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    ld_x = _matrix(x, "x", x.dtype)
    M, H = x.shape
    ld_y = 0 if y is None else _matrix(y, "y", _BF16, M, H)
    if y is None and (post or gate is not None):
        raise ValueError("a gate and the norm after the block need y")
    if not pre and (w_pre is not None or b_pre is not None):
        raise ValueError("w_pre and b_pre belong to the norm before the next block (pre=True)")
    if not post and w_post is not None:
        raise ValueError("w_post belongs to the norm after the block (post=True)")
    flags = (_PRE if pre else 0) | (_POST if post else 0) | (_F32_STREAM if x.dtype is _F32 else 0)
    groups, dtype = 1, None
    for p, grouped in ((gate, _GATE_GROUPED), (w_pre, _W_GROUPED), (b_pre, _B_GROUPED), (w_post, 0)):
        if p is None:
            continue
        if p.dtype is not dtype:
            if dtype is not None or (p.dtype is not _BF16 and p.dtype is not _F32):
                raise TypeError("the parameters must all be torch.bfloat16 or all torch.float32")
            dtype = p.dtype
        shape = p.shape
        if not p.is_cuda or not p.is_contiguous() or len(shape) not in (1, 2) or shape[-1] != H:
            raise ValueError(f"a parameter must be a contiguous GPU tensor [{H}] or [groups, {H}], got {tuple(shape)}")
        if len(shape) == 2 and shape[0] != 1:
            if not grouped or (groups != 1 and groups != shape[0]):
                raise ValueError("w_post is [H]; gate, w_pre and b_pre are [H] or share one number of groups")
            groups = shape[0]
            flags |= grouped
    if groups == 0 and M == 0:
        groups = 1   # a row of parameters for each row, of which there are none
    if groups == 0 or M % groups:
        raise ValueError(f"{M} rows are not a whole number of rows for each of {groups} groups")
    if dtype is _F32:
        flags |= _F32_PARAMS
    return NORM_KIND[kind], flags, M, H, groups, ld_x, ld_y


def _norm_forward(fn, x, y, gate, w_pre, b_pre, w_post, pre, post, res_scale, kind, eps, outs, x_out):
    k, flags, M, H, groups, ld_x, ld_y = _norm_setup(x, y, gate, w_pre, b_pre, w_post, pre, post, kind)
    _same_device(x, y, gate, w_pre, b_pre, w_post)
    if y is None:
        if x_out is not None or res_scale != 1.0:
            raise ValueError("without y, x' is x itself: no x_out and res_scale 1")
        ld_xo = 0
    elif x_out is None:
        x_out, ld_xo = _empty(x, (M, H), x.dtype), H if M > 1 else _one_row(H)
    else:
        _same_device(x, x_out)
        ld_xo = _matrix(x_out, "x_out", x.dtype, M, H)
    stats = x.new_empty((M, 4), dtype=_F32)
    _call(fn, k, flags, M, H, groups, _ptr(x), ld_x, _ptr(y), ld_y, _ptr(gate), _ptr(w_pre), _ptr(b_pre),
          _ptr(w_post), res_scale, eps, _ptr(x_out), ld_xo, *outs, _ptr(stats), _stream(x))
    return x if y is None else x_out, stats


def glu_block_norm(x, y=None, *, gate=None, w_pre=None, b_pre=None, w_post=None, pre=True, post=False,
                   res_scale=1.0, kind="rms", eps=1e-6, x_out=None, out=None):
    """x' = res_scale x + gate * N(y) w_post (post=True; else gate * y) and h = N(x') w_pre +
    b_pre (pre=True), N the rms or layer norm of a row: (x', h, stats).  Without y, x' is x
    itself.  gate, w_pre, b_pre: [H], or [groups, H] with one row per M / groups rows of x.
    stats is what glu_block_norm_bwd needs."""
    h, ld_h = out, 0
    if not pre:
        if out is not None:
            raise ValueError("out is the output of the norm before the next block (pre=True)")
        h = x.new_empty((0,), dtype=_BF16)
    elif out is None:
        h = _empty(x, x.shape, _BF16)
        ld_h = x.shape[-1] if x.shape[0] > 1 else _one_row(x.shape[-1])
    else:
        _same_device(x, out)
        ld_h = _matrix(out, "out", _BF16, *x.shape)
    x_out, stats = _norm_forward("glu_block_norm", x, y, gate, w_pre, b_pre, w_post, pre, post, res_scale, kind, eps,
                                 (_ptr(h), ld_h), x_out)
    return x_out, h, stats


def glu_block_norm_mxfp8(x, y=None, *, gate=None, w_pre=None, b_pre=None, w_post=None, post=False, res_scale=1.0,
                         kind="rms", eps=1e-6, x_out=None, out=None):
    """glu_block_norm with h quantized MXFP8 rowwise: (x', q [M, H], s [M, H/32], stats); q and
    s are the xq and xs of glu_gemm."""
    from . import _byte_buffer
    if x.dim() != 2:
        raise ValueError("x must be a 2-D tensor with unit column stride (no silent copies)")
    M, H = x.shape
    if out is not None:
        q, s = out
        _byte_buffer(q, "q", M * H)
        _byte_buffer(s, "s", M * (H // 32))
    else:
        q = x.new_empty((M, H), dtype=torch.uint8)
        s = x.new_empty((M, H // 32), dtype=torch.uint8)
    x_out, stats = _norm_forward("glu_block_norm_mxfp8", x, y, gate, w_pre, b_pre, w_post, True, post, res_scale,
                                 kind, eps, (_ptr(q), _ptr(s)), x_out)
    return x_out, q, s, stats


def glu_block_norm_bwd(x, y, stats, dx_out, dh, *, gate=None, w_pre=None, b_pre=None, w_post=None, pre=True,
                       post=False, res_scale=1.0, kind="rms", eps=1e-6):
    """Gradients of glu_block_norm from those of x' (dx_out, or None for zero) and of h (dh, None
    when pre=False): (dx, dy, dgate, dw_post, dw_pre, db_pre), each in its operand's type and
    shape and zero-sized where that operand is absent.  The other arguments are the
    forward's (b_pre gives only its shape; eps is in stats)."""
    k, flags, M, H, groups, ld_x, ld_y = _norm_setup(x, y, gate, w_pre, b_pre, w_post, pre, post, kind)
    _like(stats, "stats", _F32, (M, 4))
    if pre != (dh is not None):
        raise ValueError("dh is the gradient of h: given exactly when pre=True")
    if y is None and res_scale != 1.0:
        raise ValueError("without y, x' is x itself: res_scale 1")
    _same_device(x, y, stats, dx_out, dh, gate, w_pre, b_pre, w_post)
    ld_dxo = 0 if dx_out is None else _matrix(dx_out, "dx_out", x.dtype, M, H)
    ld_dh = 0 if dh is None else _matrix(dh, "dh", _BF16, M, H)
    dx = _empty(x, (M, H), x.dtype)
    dy = x.new_empty((0,), dtype=_BF16) if y is None else _empty(y, (M, H), _BF16)

    def grad_of(p):
        return x.new_empty((0,), dtype=_BF16) if p is None else torch.empty_like(p)

    dgate, dw_post, dw_pre, db_pre = grad_of(gate), grad_of(w_post), grad_of(w_pre), grad_of(b_pre)
    nbytes = _size("glu_block_norm_bwd_work_bytes", M, H, groups)
    work, ld = x.new_empty((max(nbytes, 0),), dtype=torch.uint8), H if M > 1 else _one_row(H)
    _call("glu_block_norm_bwd", k, flags, M, H, groups, _ptr(x), ld_x, _ptr(y), ld_y, _ptr(stats), _ptr(dx_out),
          ld_dxo, _ptr(dh), ld_dh, _ptr(gate), _ptr(w_pre), _ptr(w_post), res_scale, _ptr(dx), ld, _ptr(dy),
          ld, _ptr(dgate), _ptr(dw_pre), _ptr(db_pre),
          _ptr(dw_post), _ptr(work), nbytes, _stream(x))
    return dx, dy, dgate, dw_post, dw_pre, db_pre


# ---- linear products -------------------------------------------------------------------------

def _linear_setup(x, w, offsets, act):
    if act not in LINEAR_ACT:
        raise ValueError(f"act must be one of {sorted(LINEAR_ACT)}")
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K], or [groups, N, K] with offsets")
    if (w.dim() == 3) != (offsets is not None):
        raise ValueError("offsets go with w [groups, N, K], and only with it")
    N, K = w.shape[-2:]
    groups = w.shape[0] if w.dim() == 3 else 1
    _like(w, "w", _BF16, w.shape)
    ld_x = _matrix(x, "x", _BF16, None, K)
    if offsets is not None:
        _like(offsets, "offsets", _I32, (groups + 1,))
    return x.shape[0], N, K, groups, ld_x


def glu_linear(x, w, bias=None, residual=None, *, act="none", offsets=None, save_pre=False, out=None):
    """y = act(x W^T + bias) + residual, [M, N].  w is [N, K], or [groups, N, K] with int32
    offsets [groups + 1]: rows offsets[e] .. offsets[e + 1] - 1 of x go through w[e], bias[e], and rows
    of no group give zeros, without bias or residual.
    save_pre=True returns (y, pre), pre the FP16 pre-activation that glu_linear_bwd takes."""
    M, N, K, groups, ld_x = _linear_setup(x, w, offsets, act)
    if bias is not None:
        _like(bias, "bias", _BF16, w.shape[:-1])
    _same_device(x, w, bias, residual, offsets, out)
    ld_res = 0 if residual is None else _matrix(residual, "residual", _BF16, M, N)
    if out is None:
        y, ld_y = x.new_empty((M, N)), N
    else:
        y, ld_y = out, _matrix(out, "out", _BF16, M, N)
    pre = x.new_empty((M, N), dtype=torch.float16) if save_pre else None
    nbytes = _size("glu_linear_work_bytes", M, N, K, groups, int(offsets is not None))
    work = x.new_empty((nbytes,), dtype=torch.uint8) if nbytes > 0 else None
    _launch(x, "glu_linear", LINEAR_ACT[act], M, N, K, groups, _ptr(offsets), _ptr(x), ld_x, _ptr(w), _ptr(bias),
            _ptr(residual), ld_res, _ptr(y), ld_y, _ptr(pre), _ptr(work), nbytes)
    return (y, pre) if save_pre else y


def glu_linear_bwd(dy, x, w, *, pre=None, act="none", offsets=None, bias=False, need_dx=True, need_dw=True):
    """Gradients of glu_linear: (dx [M, K], dw like w, db [N] or [groups, N]).  pre is the
    forward's (act other than "none"); bias=True asks for db.  What is not wanted comes back
    zero-sized.  The residual's gradient is dy, with offsets zero in rows of no group."""
    M, N, K, groups, ld_x = _linear_setup(x, w, offsets, act)
    ld_dy = _matrix(dy, "dy", _BF16, M, N)
    a = LINEAR_ACT[act]
    if (a != 0) != (pre is not None):
        raise ValueError('pre goes with an act other than "none", and only with it')
    if pre is not None:
        _like(pre, "pre", torch.float16, (M, N))
    _same_device(x, w, dy, pre, offsets)
    dx = _empty(x, (M, K), _BF16) if need_dx else x.new_empty((0,))
    dw = torch.empty_like(w) if need_dw else x.new_empty((0,))
    db = x.new_empty(w.shape[:-1] if bias else (0,))
    nbytes = _size("glu_linear_bwd_work_bytes", a, M, N, K, groups, int(offsets is not None), int(bias))
    work = x.new_empty((nbytes,), dtype=torch.uint8) if nbytes > 0 else None
    _launch(x, "glu_linear_bwd", a, M, N, K, groups, _ptr(offsets), _ptr(dy), ld_dy, _ptr(x), ld_x, _ptr(w), _ptr(pre),
            _ptr(dx), K, _ptr(dw), _ptr(db), _ptr(work), nbytes)
    return dx, dw, db


# ---- expert routing --------------------------------------------------------------------------

def glu_moe_sort(ids, experts):
    """Places of a stable sort by expert: (rows int32 like ids, offsets int32 [experts + 1]).
    ids [tokens, choices] is int32 or int64; a number outside 0 .. experts - 1 is a dropped
    choice and gets row -1."""
    if ids.dtype not in (_I32, torch.int64):
        raise TypeError(f"ids must be torch.int32 or torch.int64, got {ids.dtype}")
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, choices]")
    _like(ids, "ids", ids.dtype, ids.shape)
    T, k = ids.shape
    rows = _empty(ids, (T, k), _I32)
    offsets = ids.new_empty((experts + 1,), dtype=_I32)
    nbytes = _size("glu_moe_sort_work_bytes", T, k, experts)
    work = ids.new_empty((nbytes,), dtype=torch.uint8) if nbytes > 0 else None
    _call("glu_moe_sort", T, k, experts, _ptr(ids), ids.element_size(), _ptr(rows), _ptr(offsets), _ptr(work), nbytes,
          _stream(ids))
    return rows, offsets


def _routing(rows, offsets=None):
    if rows.dim() != 2:
        raise ValueError("rows must be [tokens, choices]")
    _like(rows, "rows", _I32, rows.shape)
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("offsets must be [experts + 1]")
        _like(offsets, "offsets", _I32, offsets.shape)
    return rows.shape


def glu_moe_permute(x, rows, offsets, *, out=None):
    """xs [tokens * choices, H] with xs[rows[t, j]] = x[t] and zero rows past offsets[-1]; x may
    have any dtype (codes and scales of quantized tokens too)."""
    T, k = _routing(rows, offsets)
    ld_x = _matrix(x, "x", x.dtype)
    M, H = x.shape
    if M != T:
        raise ValueError(f"x must have {T} rows, got {M}")
    _same_device(x, rows, offsets, out)
    xs = out if out is not None else x.new_empty((T * k, H))
    ld_xs = _matrix(xs, "out", x.dtype, T * k, H)
    e = x.element_size()
    _call("glu_moe_permute", T, k, offsets.numel() - 1, H * e, _ptr(x), ld_x * e, _ptr(rows),
          _ptr(offsets), _ptr(xs), ld_xs * e, _stream(x))
    return xs


def glu_moe_combine(y, rows, weights=None, residual=None, *, out=None):
    """out[t] = residual[t] + sum over j of weights[t, j] y[rows[t, j]], dropped choices left out:
    [tokens, H].  weights float32 like rows, or None for ones (the gradient of permute)."""
    T, k = _routing(rows)
    ld_y = _matrix(y, "y", _BF16, T * k)
    H = y.shape[1]
    if weights is not None:
        _like(weights, "weights", _F32, (T, k))
    _same_device(y, rows, weights, residual, out)
    ld_res = 0 if residual is None else _matrix(residual, "residual", _BF16, T, H)
    o = out if out is not None else y.new_empty((T, H))
    _call("glu_moe_combine", T, k, H, _ptr(y), ld_y, _ptr(rows), _ptr(weights), _ptr(residual), ld_res, _ptr(o),
          _matrix(o, "out", _BF16, T, H), _stream(y))
    return o


def glu_moe_combine_bwd(dout, y, rows, weights, offsets):
    """Gradients of glu_moe_combine: (dy like y, zero rows past offsets[-1]; dweights float32,
    0 for dropped choices).  The residual's gradient is dout."""
    T, k = _routing(rows, offsets)
    ld_y = _matrix(y, "y", _BF16, T * k)
    H = y.shape[1]
    ld_d = _matrix(dout, "dout", _BF16, T, H)
    _like(weights, "weights", _F32, (T, k))
    _same_device(y, dout, rows, weights, offsets)
    dy = _empty(y, (T * k, H), _BF16)
    dw = torch.empty_like(weights)
    _call("glu_moe_combine_bwd", T, k, H, offsets.numel() - 1, _ptr(dout), ld_d, _ptr(y), ld_y, _ptr(rows),
          _ptr(weights), _ptr(offsets), _ptr(dy), _one_row(H) if T * k == 1 else H, _ptr(dw), _stream(y))
    return dy, dw

"""torch custom ops over the library's entry points (framework integration).

The "Add swiglu + MXFP8 fused CuTe DSL kernel" page (API) exposes its kernel as a torch op
that torch.compile keeps whole; these ops do the same for the MI355X kernels:

  torch.ops.glu_mx.glu(gate, up, act, layout)                          -> h
  torch.ops.glu_mx.glu_backward(gate, up, dh, act, layout)             -> (da, db) or (d, empty)
  torch.ops.glu_mx.glu_mxfp8(gate, up, act, layout, rowwise, colwise, swizzled)
                                                                       -> (q_row, q_col, s_row, s_col)
  torch.ops.glu_mx.glu_backward_mxfp8(gate, up, dh, act, rowwise, colwise, swizzled)
                                                                       -> (q_row, q_col, s_row, s_col)
  torch.ops.glu_mx.glu_nvfp4(x, up, act, layout, sf_layout)            -> (q, sf)
  torch.ops.glu_mx.glu_backward_nvfp4(gate, up, dh, act, sf_layout)    -> (q, sf)
  torch.ops.glu_mx.glu_amax(gate, up, act, layout)                     -> amax [1]
  torch.ops.glu_mx.glu_nvfp4_gs(x, up, amax, act, layout, sf_layout)   -> (q, sf)
  torch.ops.glu_mx.glu_gemm(xq, xs, wq, ws, act, fmt, w_layout)        -> h
  torch.ops.glu_mx.glu_gemm_mxfp8(xq, xs, wq, ws, act, fmt, w_layout)  -> (q_row, s_row)
  torch.ops.glu_mx.glu_gemm_nvfp4(xq, xs, wq, ws, act, sf_layout, fmt, w_layout) -> (q, sf)
  torch.ops.glu_mx.glu_gemm_nvfp4_gs(xq, xs, wq, ws, amax, act, sf_layout, fmt, w_layout) -> (q, sf)
  torch.ops.glu_mx.block_norm(x, y, gate, w_pre, b_pre, w_post, post, res_scale, kind, eps)
                                                                       -> (x_out, h, stats)
  torch.ops.glu_mx.block_norm_backward(x, y, stats, dx_out, dh, gate, w_pre, b_pre, w_post, post,
                                       res_scale, kind)  -> (dx, dy, dgate, dw_post, dw_pre, db_pre)
  torch.ops.glu_mx.linear(x, w, bias, residual, offsets, act, save_pre) -> (y, pre)
  torch.ops.glu_mx.linear_backward(dy, x, w, pre, offsets, act, bias, need_dx, need_dw)
                                                                       -> (dx, dw, db)
  torch.ops.glu_mx.moe_sort(ids, experts)                              -> (rows, offsets)
  torch.ops.glu_mx.moe_permute(x, rows, offsets)                       -> xs
  torch.ops.glu_mx.moe_combine(y, rows, offsets, weights, residual)    -> out
  torch.ops.glu_mx.moe_combine_backward(dout, y, rows, weights, offsets) -> (dy, dweights)

Each real implementation is the binding function of the same name (argument marshalling;
the HIP kernels compute everything).  Each fake implementation gives the output shapes and
dtypes without touching a GPU, so FakeTensor tracing and torch.compile(fullgraph=True)
capture the ops as single graph nodes.  `glu` is differentiable: its backward is the
`glu_backward` op (the fused BF16 backward kernel); so are block_norm, linear, moe_permute (of
BF16 rows) and moe_combine, through the backward ops beside them.  The quantized ops are not
differentiable.  In the split layout `up` is the second operand; in the paired layout pass
an empty `up` (a 0-element tensor), since a custom op cannot take None for a tensor that
other layouts need.
"""
from typing import Optional, Tuple

import torch
from torch import Tensor

from . import (glu_amax as _amax, glu_bwd as _bwd, glu_bwd_mxfp8 as _bwd_mx,
               glu_bwd_nvfp4 as _bwd_nv, glu_fwd as _fwd, glu_fwd_mxfp8 as _fwd_mx,
               glu_fwd_nvfp4 as _fwd_nv, glu_fwd_nvfp4_gs as _fwd_nv_gs, glu_gemm as _gemm,
               glu_gemm_mxfp8 as _gemm_mx, glu_gemm_nvfp4 as _gemm_nv,
               glu_gemm_nvfp4_gs as _gemm_nv_gs)
from . import (glu_block_norm as _norm, glu_block_norm_bwd as _norm_bwd, glu_linear as _linear,
               glu_linear_bwd as _linear_bwd, glu_moe_combine as _combine,
               glu_moe_combine_bwd as _combine_bwd, glu_moe_permute as _permute, glu_moe_sort as _sort)

_LIB = "glu_mx"


def _up(up, layout):
    return None if layout == "paired" else up


def _width(gate, layout):
    """Per-half width N of the GLU output."""
    return gate.shape[1] // 2 if layout == "paired" else gate.shape[1]


def _mx_scale_shape(rows, cols, swizzled):
    if swizzled:
        return ((rows + 127) // 128 * 128 * ((cols // 32 + 3) // 4 * 4),)
    return (rows, cols // 32)


def _nv_scale_shape(rows, cols, sf_layout):
    if sf_layout == "128x4":
        return ((rows + 127) // 128 * 128 * ((cols // 16 + 3) // 4 * 4),)
    return (rows, cols // 16)


def _mx_fake(ref, rows, cols, rowwise, colwise, swizzled):
    u8 = dict(dtype=torch.uint8, device=ref.device)
    z = torch.empty((0,), **u8)
    return (torch.empty((rows, cols), **u8) if rowwise else z,
            torch.empty((cols, rows), **u8) if colwise else z,
            torch.empty(_mx_scale_shape(rows, cols, swizzled), **u8) if rowwise else z,
            torch.empty(_mx_scale_shape(cols, rows, swizzled), **u8) if colwise else z)


# ---- BF16 GLU, differentiable -------------------------------------------------------

@torch.library.custom_op(f"{_LIB}::glu", mutates_args=())
def glu(gate: Tensor, up: Tensor, act: str = "swiglu", layout: str = "split") -> Tensor:
    return _fwd(gate, _up(up, layout), act=act, layout=layout)


@glu.register_fake
def _(gate, up, act="swiglu", layout="split"):
    return gate.new_empty((gate.shape[0], _width(gate, layout)))


@torch.library.custom_op(f"{_LIB}::glu_backward", mutates_args=())
def glu_backward(gate: Tensor, up: Tensor, dh: Tensor, act: str = "swiglu",
                 layout: str = "split") -> Tuple[Tensor, Tensor]:
    """Split: (da, db).  Paired: (the interleaved gradient of the paired operand, empty)."""
    if layout == "paired":
        return _bwd(gate, None, dh, act=act, layout="paired"), gate.new_empty((0,))
    return _bwd(gate, up, dh, act=act)


@glu_backward.register_fake
def _(gate, up, dh, act="swiglu", layout="split"):
    if layout == "paired":
        return gate.new_empty(gate.shape), gate.new_empty((0,))
    return gate.new_empty(gate.shape), up.new_empty(up.shape)


def _glu_setup(ctx, inputs, output):
    gate, up, act, layout = inputs
    ctx.save_for_backward(gate, up)
    ctx.act, ctx.layout = act, layout


def _glu_grad(ctx, dh):
    gate, up = ctx.saved_tensors
    # the binding takes unit-stride rows; autograd may hand over a broadcast gradient
    d0, d1 = glu_backward(gate, up, dh.contiguous(), ctx.act, ctx.layout)
    if ctx.layout == "paired":
        return d0, None, None, None
    return d0, d1, None, None


glu.register_autograd(_glu_grad, setup_context=_glu_setup)


# ---- fused MXFP8 --------------------------------------------------------------------

@torch.library.custom_op(f"{_LIB}::glu_mxfp8", mutates_args=())
def glu_mxfp8(gate: Tensor, up: Tensor, act: str = "swiglu", layout: str = "split",
              rowwise: bool = True, colwise: bool = False,
              swizzled: bool = False) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    return _fwd_mx(gate, _up(up, layout), act=act, layout=layout, rowwise=rowwise,
                   colwise=colwise, swizzled=swizzled)


@glu_mxfp8.register_fake
def _(gate, up, act="swiglu", layout="split", rowwise=True, colwise=False, swizzled=False):
    return _mx_fake(gate, gate.shape[0], _width(gate, layout), rowwise, colwise, swizzled)


@torch.library.custom_op(f"{_LIB}::glu_backward_mxfp8", mutates_args=())
def glu_backward_mxfp8(gate: Tensor, up: Tensor, dh: Tensor, act: str = "swiglu",
                       rowwise: bool = True, colwise: bool = False,
                       swizzled: bool = False) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    return _bwd_mx(gate, up, dh, act=act, rowwise=rowwise, colwise=colwise, swizzled=swizzled)


@glu_backward_mxfp8.register_fake
def _(gate, up, dh, act="swiglu", rowwise=True, colwise=False, swizzled=False):
    return _mx_fake(gate, gate.shape[0], 2 * gate.shape[1], rowwise, colwise, swizzled)


# ---- fused NVFP4 --------------------------------------------------------------------

@torch.library.custom_op(f"{_LIB}::glu_nvfp4", mutates_args=())
def glu_nvfp4(x: Tensor, up: Tensor, act: str = "geglu", layout: str = "paired",
              sf_layout: str = "rowmajor") -> Tuple[Tensor, Tensor]:
    return _fwd_nv(x, _up(up, layout), act=act, layout=layout, sf_layout=sf_layout)


@glu_nvfp4.register_fake
def _(x, up, act="geglu", layout="paired", sf_layout="rowmajor"):
    M, H = x.shape[0], _width(x, layout)
    return (x.new_empty((M, H // 2), dtype=torch.uint8),
            x.new_empty(_nv_scale_shape(M, H, sf_layout), dtype=torch.uint8))


@torch.library.custom_op(f"{_LIB}::glu_backward_nvfp4", mutates_args=())
def glu_backward_nvfp4(gate: Tensor, up: Tensor, dh: Tensor, act: str = "swiglu",
                       sf_layout: str = "rowmajor") -> Tuple[Tensor, Tensor]:
    return _bwd_nv(gate, up, dh, act=act, sf_layout=sf_layout)


@glu_backward_nvfp4.register_fake
def _(gate, up, dh, act="swiglu", sf_layout="rowmajor"):
    M, N = gate.shape
    return (gate.new_empty((M, N), dtype=torch.uint8),
            gate.new_empty(_nv_scale_shape(M, 2 * N, sf_layout), dtype=torch.uint8))


@torch.library.custom_op(f"{_LIB}::glu_amax", mutates_args=())
def glu_amax(gate: Tensor, up: Tensor, act: str = "swiglu", layout: str = "split") -> Tensor:
    return _amax(gate, _up(up, layout), act=act, layout=layout)


@glu_amax.register_fake
def _(gate, up, act="swiglu", layout="split"):
    return gate.new_empty((1,), dtype=torch.float32)


@torch.library.custom_op(f"{_LIB}::glu_nvfp4_gs", mutates_args=())
def glu_nvfp4_gs(x: Tensor, up: Tensor, amax: Tensor, act: str = "geglu", layout: str = "paired",
                 sf_layout: str = "rowmajor") -> Tuple[Tensor, Tensor]:
    return _fwd_nv_gs(x, _up(up, layout), amax=amax, act=act, layout=layout, sf_layout=sf_layout)


@glu_nvfp4_gs.register_fake
def _(x, up, amax, act="geglu", layout="paired", sf_layout="rowmajor"):
    M, H = x.shape[0], _width(x, layout)
    return (x.new_empty((M, H // 2), dtype=torch.uint8),
            x.new_empty(_nv_scale_shape(M, H, sf_layout), dtype=torch.uint8))


# ---- merged gate/up block-scaled GEMM with the GLU epilogue ---------------------------
# xq [M, K] codes (fmt "mxfp8": E4M3, one per byte; "mxfp4": E2M1, [M, K/2] packed), xs [M, K/32]
# E8M0 scales, wq [2N, K] (rows [W_gate | W_up], or gate0, up0, ... with w_layout "paired"),
# ws [2N, K/32]

@torch.library.custom_op(f"{_LIB}::glu_gemm", mutates_args=())
def glu_gemm(xq: Tensor, xs: Tensor, wq: Tensor, ws: Tensor, act: str = "swiglu", fmt: str = "mxfp8",
             w_layout: str = "split") -> Tensor:
    return _gemm(xq, xs, wq, ws, act=act, fmt=fmt, w_layout=w_layout)


@glu_gemm.register_fake
def _(xq, xs, wq, ws, act="swiglu", fmt="mxfp8", w_layout="split"):
    return xq.new_empty((xq.shape[0], wq.shape[0] // 2), dtype=torch.bfloat16)


@torch.library.custom_op(f"{_LIB}::glu_gemm_mxfp8", mutates_args=())
def glu_gemm_mxfp8(xq: Tensor, xs: Tensor, wq: Tensor, ws: Tensor, act: str = "swiglu",
                   fmt: str = "mxfp8", w_layout: str = "split") -> Tuple[Tensor, Tensor]:
    return _gemm_mx(xq, xs, wq, ws, act=act, fmt=fmt, w_layout=w_layout)


@glu_gemm_mxfp8.register_fake
def _(xq, xs, wq, ws, act="swiglu", fmt="mxfp8", w_layout="split"):
    M, N = xq.shape[0], wq.shape[0] // 2
    return xq.new_empty((M, N), dtype=torch.uint8), xq.new_empty((M, N // 32), dtype=torch.uint8)


@torch.library.custom_op(f"{_LIB}::glu_gemm_nvfp4", mutates_args=())
def glu_gemm_nvfp4(xq: Tensor, xs: Tensor, wq: Tensor, ws: Tensor, act: str = "geglu",
                   sf_layout: str = "rowmajor", fmt: str = "mxfp8",
                   w_layout: str = "split") -> Tuple[Tensor, Tensor]:
    return _gemm_nv(xq, xs, wq, ws, act=act, sf_layout=sf_layout, fmt=fmt, w_layout=w_layout)


@glu_gemm_nvfp4.register_fake
def _(xq, xs, wq, ws, act="geglu", sf_layout="rowmajor", fmt="mxfp8", w_layout="split"):
    M, N = xq.shape[0], wq.shape[0] // 2
    return (xq.new_empty((M, N // 2), dtype=torch.uint8),
            xq.new_empty(_nv_scale_shape(M, N, sf_layout), dtype=torch.uint8))


@torch.library.custom_op(f"{_LIB}::glu_gemm_nvfp4_gs", mutates_args=())
def glu_gemm_nvfp4_gs(xq: Tensor, xs: Tensor, wq: Tensor, ws: Tensor, amax: Tensor,
                      act: str = "geglu", sf_layout: str = "rowmajor", fmt: str = "mxfp8",
                      w_layout: str = "split") -> Tuple[Tensor, Tensor]:
    return _gemm_nv_gs(xq, xs, wq, ws, amax=amax, act=act, sf_layout=sf_layout, fmt=fmt, w_layout=w_layout)


@glu_gemm_nvfp4_gs.register_fake
def _(xq, xs, wq, ws, amax, act="geglu", sf_layout="rowmajor", fmt="mxfp8", w_layout="split"):
    M, N = xq.shape[0], wq.shape[0] // 2
    return (xq.new_empty((M, N // 2), dtype=torch.uint8),
            xq.new_empty(_nv_scale_shape(M, N, sf_layout), dtype=torch.uint8))


def _incoming(grad):
    """A gradient as the kernels take it: contiguous, from a 16-byte boundary.  That of one part of a
    concatenation is a view that starts where the part does."""
    grad = grad.contiguous()
    return grad.clone() if grad.storage_offset() * grad.element_size() % 16 else grad


# ---- block norms, differentiable ------------------------------------------------------
# Without y, x' is x itself and x_out comes back zero-sized (an op may not return its input).
# stats is for the backward and has no gradient.

@torch.library.custom_op(f"{_LIB}::block_norm", mutates_args=())
def block_norm(x: Tensor, y: Optional[Tensor] = None, gate: Optional[Tensor] = None,
               w_pre: Optional[Tensor] = None, b_pre: Optional[Tensor] = None, w_post: Optional[Tensor] = None,
               post: bool = False, res_scale: float = 1.0, kind: str = "rms",
               eps: float = 1e-6) -> Tuple[Tensor, Tensor, Tensor]:
    x_out, h, stats = _norm(x, y, gate=gate, w_pre=w_pre, b_pre=b_pre, w_post=w_post, post=post,
                            res_scale=res_scale, kind=kind, eps=eps)
    return x.new_empty((0,)) if y is None else x_out, h, stats


@block_norm.register_fake
def _(x, y=None, gate=None, w_pre=None, b_pre=None, w_post=None, post=False, res_scale=1.0, kind="rms", eps=1e-6):
    return (x.new_empty((0,) if y is None else x.shape), x.new_empty(x.shape, dtype=torch.bfloat16),
            x.new_empty((x.shape[0], 4), dtype=torch.float32))


@torch.library.custom_op(f"{_LIB}::block_norm_backward", mutates_args=())
def block_norm_backward(x: Tensor, y: Optional[Tensor], stats: Tensor, dx_out: Optional[Tensor], dh: Tensor,
                        gate: Optional[Tensor], w_pre: Optional[Tensor], b_pre: Optional[Tensor],
                        w_post: Optional[Tensor], post: bool, res_scale: float,
                        kind: str) -> Tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor]:
    return _norm_bwd(x, y, stats, dx_out, dh, gate=gate, w_pre=w_pre, b_pre=b_pre, w_post=w_post, post=post,
                     res_scale=res_scale, kind=kind)


@block_norm_backward.register_fake
def _(x, y, stats, dx_out, dh, gate, w_pre, b_pre, w_post, post, res_scale, kind):
    def like(t):
        return x.new_empty((0,), dtype=torch.bfloat16) if t is None else t.new_empty(t.shape)
    return x.new_empty(x.shape), like(y), like(gate), like(w_post), like(w_pre), like(b_pre)


def _norm_setup(ctx, inputs, output):
    x, y, gate, w_pre, b_pre, w_post, ctx.post, ctx.res_scale, ctx.kind, _ = inputs
    ctx.save_for_backward(x, y, output[2], gate, w_pre, b_pre, w_post)
    ctx.mark_non_differentiable(output[2])


def _norm_grad(ctx, dx_out, dh, _):
    x, y, stats, gate, w_pre, b_pre, w_post = ctx.saved_tensors
    dx, dy, dgate, dw_post, dw_pre, db_pre = block_norm_backward(
        x, y, stats, None if y is None else _incoming(dx_out), _incoming(dh), gate, w_pre, b_pre, w_post,
        ctx.post, ctx.res_scale, ctx.kind)
    grads = [g if t is not None else None for g, t in ((dy, y), (dgate, gate), (dw_pre, w_pre), (db_pre, b_pre),
                                                      (dw_post, w_post))]
    return (dx, *grads, None, None, None, None)


block_norm.register_autograd(_norm_grad, setup_context=_norm_setup)


# ---- linear products, differentiable ----------------------------------------------------
# pre is the pre-activation the backward needs, zero-sized when act is "none" or save_pre is off
# (then only y's residual has a gradient with an act).  It has no gradient of its own.

@torch.library.custom_op(f"{_LIB}::linear", mutates_args=())
def linear(x: Tensor, w: Tensor, bias: Optional[Tensor] = None, residual: Optional[Tensor] = None,
           offsets: Optional[Tensor] = None, act: str = "none", save_pre: bool = True) -> Tuple[Tensor, Tensor]:
    if act != "none" and save_pre:
        return _linear(x, w, bias, residual, act=act, offsets=offsets, save_pre=True)
    return _linear(x, w, bias, residual, act=act, offsets=offsets), x.new_empty((0,), dtype=torch.float16)


@linear.register_fake
def _(x, w, bias=None, residual=None, offsets=None, act="none", save_pre=True):
    shape = (x.shape[0], w.shape[-2])
    return x.new_empty(shape), x.new_empty(shape if act != "none" and save_pre else (0,), dtype=torch.float16)


@torch.library.custom_op(f"{_LIB}::linear_backward", mutates_args=())
def linear_backward(dy: Tensor, x: Tensor, w: Tensor, pre: Optional[Tensor], offsets: Optional[Tensor], act: str,
                    bias: bool, need_dx: bool = True, need_dw: bool = True) -> Tuple[Tensor, Tensor, Tensor]:
    return _linear_bwd(dy, x, w, pre=pre, act=act, offsets=offsets, bias=bias, need_dx=need_dx, need_dw=need_dw)


@linear_backward.register_fake
def _(dy, x, w, pre, offsets, act, bias, need_dx=True, need_dw=True):
    return (x.new_empty(x.shape if need_dx else (0,)), w.new_empty(w.shape if need_dw else (0,)),
            w.new_empty(w.shape[:-1] if bias else (0,)))


def _linear_setup(ctx, inputs, output):
    x, w, _, _, offsets, ctx.act, save_pre = inputs
    ctx.no_pre = ctx.act != "none" and not save_pre
    ctx.save_for_backward(x, w, None if ctx.act == "none" else output[1], offsets)
    ctx.mark_non_differentiable(output[1])


def _rows_of_groups(dy, offsets):
    """The residual's gradient: dy, but zero in rows of no group, where y is zero without it."""
    if offsets is None:
        return dy
    row = torch.arange(dy.shape[0], device=dy.device)
    return dy.masked_fill(((row < offsets[0]) | (row >= offsets[-1])).unsqueeze(1), 0.0)


def _linear_grad(ctx, dy, _):
    x, w, pre, offsets = ctx.saved_tensors
    # arguments left to their defaults at the end of a call have no entry
    need_dx, need_dw, need_db, need_dres = (tuple(ctx.needs_input_grad) + (False, False))[:4]
    dy = _incoming(dy)
    dx = dw = db = None
    if need_dx or need_dw or need_db:
        if ctx.no_pre:
            raise RuntimeError("linear was called with save_pre=False: its activation has no gradient")
        dx, dw, db = linear_backward(dy, x, w, pre, offsets, ctx.act, need_db, need_dx, need_dw)
    return (dx if need_dx else None, dw if need_dw else None, db if need_db else None,
            _rows_of_groups(dy, offsets) if need_dres else None, None, None, None)


linear.register_autograd(_linear_grad, setup_context=_linear_setup)


# ---- expert routing, differentiable -----------------------------------------------------

@torch.library.custom_op(f"{_LIB}::moe_sort", mutates_args=())
def moe_sort(ids: Tensor, experts: int) -> Tuple[Tensor, Tensor]:
    return _sort(ids, experts)


@moe_sort.register_fake
def _(ids, experts):
    return ids.new_empty(ids.shape, dtype=torch.int32), ids.new_empty((experts + 1,), dtype=torch.int32)


@torch.library.custom_op(f"{_LIB}::moe_permute", mutates_args=())
def moe_permute(x: Tensor, rows: Tensor, offsets: Tensor) -> Tensor:
    return _permute(x, rows, offsets)


@moe_permute.register_fake
def _(x, rows, offsets):
    return x.new_empty((rows.shape[0] * rows.shape[1], x.shape[1]))


@torch.library.custom_op(f"{_LIB}::moe_combine", mutates_args=())
def moe_combine(y: Tensor, rows: Tensor, offsets: Tensor, weights: Optional[Tensor] = None,
                residual: Optional[Tensor] = None) -> Tensor:
    return _combine(y, rows, weights, residual)


@moe_combine.register_fake
def _(y, rows, offsets, weights=None, residual=None):
    return y.new_empty((rows.shape[0], y.shape[1]))


@torch.library.custom_op(f"{_LIB}::moe_combine_backward", mutates_args=())
def moe_combine_backward(dout: Tensor, y: Tensor, rows: Tensor, weights: Tensor,
                         offsets: Tensor) -> Tuple[Tensor, Tensor]:
    return _combine_bwd(dout, y, rows, weights, offsets)


@moe_combine_backward.register_fake
def _(dout, y, rows, weights, offsets):
    return y.new_empty(y.shape), weights.new_empty(weights.shape)


def _permute_setup(ctx, inputs, output):
    _, rows, offsets = inputs
    ctx.save_for_backward(rows, offsets)


def _permute_grad(ctx, dxs):
    rows, offsets = ctx.saved_tensors
    return moe_combine(_incoming(dxs), rows, offsets), None, None


def _combine_setup(ctx, inputs, output):
    y, rows, offsets, weights, residual = inputs
    ctx.has_residual = residual is not None
    ctx.save_for_backward(y, rows, offsets, weights)


def _combine_grad(ctx, dout):
    y, rows, offsets, weights = ctx.saved_tensors
    dout = _incoming(dout)
    dres = dout if ctx.has_residual else None
    if weights is None:
        return moe_permute(dout, rows, offsets), None, None, None, dres
    dy, dw = moe_combine_backward(dout, y, rows, weights, offsets)
    return dy, None, None, dw, dres


moe_permute.register_autograd(_permute_grad, setup_context=_permute_setup)
moe_combine.register_autograd(_combine_grad, setup_context=_combine_setup)

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
  torch.ops.glu_mx.gated_linear(x, w, bias, offsets, act, w_layout, save) -> (h, pre, extra)
  torch.ops.glu_mx.gated_linear_backward(dh, x, w, pre, extra, offsets, act, w_layout, bias, need_dx,
                                         need_dw)          -> (dx, dw, db)
  torch.ops.glu_mx.glu_ckpt(gate, up, act, layout)                     -> (h, q, s)
  torch.ops.glu_mx.glu_ckpt_backward(q, s, dh, act, layout, need_h)    -> (d, h)
  torch.ops.glu_mx.feed_forward(x, w13, w2, b13, b2, offsets, act, w_layout, save) -> (y, pre, extra)
  torch.ops.glu_mx.feed_forward_backward(dy, x, w13, w2, pre, extra, offsets, act, w_layout, bias13, bias2,
                                         need_dx, need_dw13, need_dw2) -> (dx, dw13, dw2, db13, db2)
  torch.ops.glu_mx.quant_fp8(x, rowwise, colwise)                      -> (q_row, q_col, s_row, s_col)
  torch.ops.glu_mx.glu_fp8(gate, up, act, layout, rowwise, colwise)    -> the same of act(gate) * up
  torch.ops.glu_mx.quant_fp8_weight(w, transpose)                      -> (q, s, qt, st)
  torch.ops.glu_mx.product_fp8(xq, xs, wq, ws, bias, residual, offsets, w_scales) -> y
  torch.ops.glu_mx.linear_fp8(x, w, bias, residual)                    -> (y, xq, xs, wq, ws)
  torch.ops.glu_mx.linear_fp8_backward(dy, xq, xs, wq, ws, need_dx, need_dw, bias) -> (dx, dw, db)

Each real implementation is the binding function of the same name (argument marshalling;
the HIP kernels compute everything).  Each fake implementation gives the output shapes and
dtypes without touching a GPU, so FakeTensor tracing and torch.compile(fullgraph=True)
capture the ops as single graph nodes.  `glu` is differentiable: its backward is the
`glu_backward` op (the fused BF16 backward kernel); so are block_norm, linear, moe_permute (of
BF16 rows), moe_combine, gated_linear, glu_ckpt, feed_forward and linear_fp8, through the backward
ops beside them.  glu_ckpt keeps gate and up for its backward in 8 bits, feed_forward what its `save`
says (and forms the GLU's result again instead of keeping it), linear_fp8 x and w as 8-bit codes.  The
other quantized ops are not differentiable.  In the split layout `up` is the second operand; in the paired layout pass
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
from . import (glu_bwd_ckpt as _bwd_ckpt, glu_fwd_ckpt as _fwd_ckpt, glu_fwd_fp8 as _fwd_fp8,
               glu_gated_linear as _gated, glu_gated_linear_bwd as _gated_bwd, glu_linear_fp8 as _product_fp8,
               glu_quant_fp8 as _quant_fp8, glu_quant_fp8_weight as _quant_weight)

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


# ---- gated projections, differentiable --------------------------------------------------
# pre and extra are what the backward needs of gate and up, zero-sized with save="none" (which has no
# gradient).  They have no gradient of their own.

def _kept_fake(x, N, save):
    M = x.shape[0]
    if save == "none":
        return x.new_empty((0,)), x.new_empty((0,), dtype=torch.uint8)
    if save == "bf16":
        return x.new_empty((M, 2 * N)), x.new_empty((M, N), dtype=torch.uint8)
    return (x.new_empty((M, 2 * N), dtype=torch.uint8),
            x.new_empty((M, 2 * ((N + 31) // 32)), dtype=torch.uint8))


def _no_save(save):
    if save == "none":
        raise RuntimeError('called with save="none": what the gradients need was not kept')


@torch.library.custom_op(f"{_LIB}::gated_linear", mutates_args=())
def gated_linear(x: Tensor, w: Tensor, bias: Optional[Tensor] = None, offsets: Optional[Tensor] = None,
                 act: str = "swiglu", w_layout: str = "split", save: str = "bf16") -> Tuple[Tensor, Tensor, Tensor]:
    if save == "none":
        return (_gated(x, w, bias, act=act, w_layout=w_layout, offsets=offsets), x.new_empty((0,)),
                x.new_empty((0,), dtype=torch.uint8))
    return _gated(x, w, bias, act=act, w_layout=w_layout, offsets=offsets, save=save)


@gated_linear.register_fake
def _(x, w, bias=None, offsets=None, act="swiglu", w_layout="split", save="bf16"):
    N = w.shape[-2] // 2
    return (x.new_empty((x.shape[0], N)), *_kept_fake(x, N, save))


@torch.library.custom_op(f"{_LIB}::gated_linear_backward", mutates_args=())
def gated_linear_backward(dh: Tensor, x: Tensor, w: Tensor, pre: Tensor, extra: Tensor, offsets: Optional[Tensor],
                          act: str, w_layout: str, bias: bool, need_dx: bool = True,
                          need_dw: bool = True) -> Tuple[Tensor, Tensor, Tensor]:
    return _gated_bwd(dh, x, w, pre, extra, act=act, w_layout=w_layout, offsets=offsets, bias=bias, need_dx=need_dx,
                      need_dw=need_dw)[:3]


@gated_linear_backward.register_fake
def _(dh, x, w, pre, extra, offsets, act, w_layout, bias, need_dx=True, need_dw=True):
    return (x.new_empty(x.shape if need_dx else (0,)), w.new_empty(w.shape if need_dw else (0,)),
            w.new_empty(w.shape[:-1] if bias else (0,)))


def _gated_setup(ctx, inputs, output):
    x, w, _, offsets, ctx.act, ctx.w_layout, ctx.save = inputs
    ctx.save_for_backward(x, w, offsets, output[1], output[2])
    ctx.mark_non_differentiable(output[1], output[2])


def _gated_grad(ctx, dh, *_):
    _no_save(ctx.save)
    x, w, offsets, pre, extra = ctx.saved_tensors
    need = (tuple(ctx.needs_input_grad) + (False,) * 3)[:3]
    dx, dw, db = gated_linear_backward(_incoming(dh), x, w, pre, extra, offsets, ctx.act, ctx.w_layout, need[2], need[0],
                                       need[1])
    return (*(g if n else None for g, n in zip((dx, dw, db), need)), None, None, None, None)


gated_linear.register_autograd(_gated_grad, setup_context=_gated_setup)


# ---- the GLU with 8-bit checkpoints, differentiable ---------------------------------------

@torch.library.custom_op(f"{_LIB}::glu_ckpt", mutates_args=())
def glu_ckpt(gate: Tensor, up: Tensor, act: str = "swiglu", layout: str = "split") -> Tuple[Tensor, Tensor, Tensor]:
    return _fwd_ckpt(gate, _up(up, layout), act=act, layout=layout)


@glu_ckpt.register_fake
def _(gate, up, act="swiglu", layout="split"):
    M, N = gate.shape[0], _width(gate, layout)
    return (gate.new_empty((M, N)), gate.new_empty((M, 2 * N), dtype=torch.uint8),
            gate.new_empty((M, 2 * ((N + 31) // 32)), dtype=torch.uint8))


@torch.library.custom_op(f"{_LIB}::glu_ckpt_backward", mutates_args=())
def glu_ckpt_backward(q: Tensor, s: Tensor, dh: Tensor, act: str = "swiglu", layout: str = "split",
                      need_h: bool = False) -> Tuple[Tensor, Tensor]:
    """d is [dGate | dUp] (split) or the interleaved gradient (paired)."""
    return _bwd_ckpt(q, s, dh, act=act, layout=layout, need_h=need_h)


@glu_ckpt_backward.register_fake
def _(q, s, dh, act="swiglu", layout="split", need_h=False):
    return dh.new_empty(q.shape), dh.new_empty(dh.shape if need_h else (0,))


def _ckpt_setup(ctx, inputs, output):
    ctx.act, ctx.layout = inputs[2:]
    ctx.save_for_backward(output[1], output[2])
    ctx.mark_non_differentiable(output[1], output[2])


def _ckpt_grad(ctx, dh, *_):
    q, s = ctx.saved_tensors
    d, _ = glu_ckpt_backward(q, s, _incoming(dh), ctx.act, ctx.layout)
    if ctx.layout == "paired":
        return d, None, None, None
    N = d.shape[1] // 2
    return d[:, :N], d[:, N:], None, None


glu_ckpt.register_autograd(_ckpt_grad, setup_context=_ckpt_setup)


# ---- a gated feed-forward block, differentiable --------------------------------------------
# y = (act(x Wg^T + bg) * (x Wu^T + bu)) W2^T + b2.  The GLU's result is not kept: the backward forms it
# again from gate and up as kept (save "bf16" or "mxfp8"), in the pass that forms their gradients.

@torch.library.custom_op(f"{_LIB}::feed_forward", mutates_args=())
def feed_forward(x: Tensor, w13: Tensor, w2: Tensor, b13: Optional[Tensor] = None, b2: Optional[Tensor] = None,
                 offsets: Optional[Tensor] = None, act: str = "swiglu", w_layout: str = "split",
                 save: str = "mxfp8") -> Tuple[Tensor, Tensor, Tensor]:
    h, pre, extra = gated_linear(x, w13, b13, offsets, act, w_layout, save)
    return _linear(h, w2, b2, offsets=offsets), pre, extra


@feed_forward.register_fake
def _(x, w13, w2, b13=None, b2=None, offsets=None, act="swiglu", w_layout="split", save="mxfp8"):
    return (x.new_empty((x.shape[0], w2.shape[-2])), *_kept_fake(x, w13.shape[-2] // 2, save))


@torch.library.custom_op(f"{_LIB}::feed_forward_backward", mutates_args=())
def feed_forward_backward(dy: Tensor, x: Tensor, w13: Tensor, w2: Tensor, pre: Tensor, extra: Tensor,
                          offsets: Optional[Tensor], act: str, w_layout: str, bias13: bool, bias2: bool,
                          need_dx: bool = True, need_dw13: bool = True,
                          need_dw2: bool = True) -> Tuple[Tensor, Tensor, Tensor, Tensor, Tensor]:
    dx, dw13, dw2, db13, db2 = (x.new_empty((0,)) for _ in range(5))
    first = need_dx or need_dw13 or bias13   # gradients of the projections
    M, N = x.shape[0], w2.shape[-1]
    # the calls for dh and db2 read no h
    dh = h = x.new_empty((M, N))
    if first:
        dh = _linear_bwd(dy, h, w2, offsets=offsets, need_dw=False)[0]
    if first or need_dw2:
        dx, dw13, db13, h = _gated_bwd(dh, x, w13, pre, extra, act=act, w_layout=w_layout, offsets=offsets, bias=bias13,
                                       need_dx=need_dx, need_dw=need_dw13, need_h=need_dw2)
    if need_dw2 or bias2:
        _, dw2, db2 = _linear_bwd(dy, h if need_dw2 else dh, w2, offsets=offsets, bias=bias2, need_dx=False, need_dw=need_dw2)
    return dx, dw13, dw2, db13, db2


@feed_forward_backward.register_fake
def _(dy, x, w13, w2, pre, extra, offsets, act, w_layout, bias13, bias2, need_dx=True, need_dw13=True, need_dw2=True):
    def of(t, wanted, shape):
        return t.new_empty(shape if wanted else (0,))
    return (of(x, need_dx, x.shape), of(w13, need_dw13, w13.shape), of(w2, need_dw2, w2.shape),
            of(w13, bias13, w13.shape[:-1]), of(w2, bias2, w2.shape[:-1]))


def _ffn_setup(ctx, inputs, output):
    x, w13, w2, _, _, offsets, ctx.act, ctx.w_layout, ctx.save = inputs
    ctx.save_for_backward(x, w13, w2, offsets, output[1], output[2])
    ctx.mark_non_differentiable(output[1], output[2])


def _ffn_grad(ctx, dy, *_):
    _no_save(ctx.save)
    x, w13, w2, offsets, pre, extra = ctx.saved_tensors
    need = (tuple(ctx.needs_input_grad) + (False,) * 5)[:5]
    dx, dw13, dw2, db13, db2 = feed_forward_backward(_incoming(dy), x, w13, w2, pre, extra, offsets, ctx.act, ctx.w_layout,
                                                     need[3], need[4], need[0], need[1], need[2])
    return (*(g if n else None for g, n in zip((dx, dw13, dw2, db13, db2), need)), None, None, None, None)


feed_forward.register_autograd(_ffn_grad, setup_context=_ffn_setup)


# ---- 8-bit floating point with a scale for each 128 -----------------------------------------

def _fp8_fake(ref, M, N, rowwise, colwise):
    def pair(on, rows, cols):
        if not on:
            return ref.new_empty((0,), dtype=torch.uint8), ref.new_empty((0,), dtype=torch.float32)
        return (ref.new_empty((rows, (cols + 15) // 16 * 16), dtype=torch.uint8),
                ref.new_empty(((cols + 127) // 128, rows), dtype=torch.float32))
    (q_row, s_row), (q_col, s_col) = pair(rowwise, M, N), pair(colwise, N, M)
    return q_row, q_col, s_row, s_col


@torch.library.custom_op(f"{_LIB}::quant_fp8", mutates_args=())
def quant_fp8(x: Tensor, rowwise: bool = True, colwise: bool = False) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    return _quant_fp8(x, rowwise=rowwise, colwise=colwise)


@quant_fp8.register_fake
def _(x, rowwise=True, colwise=False):
    return _fp8_fake(x, x.shape[0], x.shape[1], rowwise, colwise)


@torch.library.custom_op(f"{_LIB}::glu_fp8", mutates_args=())
def glu_fp8(gate: Tensor, up: Tensor, act: str = "swiglu", layout: str = "split", rowwise: bool = True,
            colwise: bool = False) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    return _fwd_fp8(gate, _up(up, layout), act=act, layout=layout, rowwise=rowwise, colwise=colwise)


@glu_fp8.register_fake
def _(gate, up, act="swiglu", layout="split", rowwise=True, colwise=False):
    return _fp8_fake(gate, gate.shape[0], _width(gate, layout), rowwise, colwise)


def _weight_fake(w, n, k):
    lead = w.shape[:-2]
    return (w.new_empty((*lead, n, (k + 15) // 16 * 16), dtype=torch.uint8),
            w.new_empty((*lead, (n + 127) // 128, (k + 127) // 128), dtype=torch.float32))


@torch.library.custom_op(f"{_LIB}::quant_fp8_weight", mutates_args=())
def quant_fp8_weight(w: Tensor, transpose: bool = False) -> Tuple[Tensor, Tensor, Tensor, Tensor]:
    return _quant_weight(w, transpose=transpose)


@quant_fp8_weight.register_fake
def _(w, transpose=False):
    n, k = w.shape[-2:]
    none = (w.new_empty((0,), dtype=torch.uint8), w.new_empty((0,), dtype=torch.float32))
    return (*_weight_fake(w, n, k), *(_weight_fake(w, k, n) if transpose else none))


@torch.library.custom_op(f"{_LIB}::product_fp8", mutates_args=())
def product_fp8(xq: Tensor, xs: Tensor, wq: Tensor, ws: Tensor, bias: Optional[Tensor] = None,
                residual: Optional[Tensor] = None, offsets: Optional[Tensor] = None, w_scales: str = "block") -> Tensor:
    return _product_fp8(xq, xs, wq, ws, bias, residual, w_scales=w_scales, offsets=offsets)


@product_fp8.register_fake
def _(xq, xs, wq, ws, bias=None, residual=None, offsets=None, w_scales="block"):
    return xq.new_empty((xq.shape[0], wq.shape[-2]), dtype=torch.bfloat16)


# A linear layer whose three products run in 8 bits.  For the backward it keeps x quantized along its rows'
# number (colwise) and W transposed, both as codes.  The gradients are those of the product at what the
# codes of x and W stand for, with dy quantized too; the bias's is the sum of dy, the residual's dy itself.
# W's gradient sums over the rows of x, of which the product takes _MAX_ROW_SUM: a call that will want it of
# more rows is refused when it is made, not in its backward.

_MAX_ROW_SUM = 1 << 22


@torch.library.custom_op(f"{_LIB}::linear_fp8", mutates_args=())
def linear_fp8(x: Tensor, w: Tensor, bias: Optional[Tensor] = None,
               residual: Optional[Tensor] = None) -> Tuple[Tensor, Tensor, Tensor, Tensor, Tensor]:
    q_row, q_col, s_row, s_col = _quant_fp8(x, rowwise=True, colwise=True)
    wq, ws, wt, wts = _quant_weight(w, transpose=True)
    return _product_fp8(q_row, s_row, wq, ws, bias, residual), q_col, s_col, wt, wts


@linear_fp8.register_fake
def _(x, w, bias=None, residual=None):
    _, q_col, _, s_col = _fp8_fake(x, x.shape[0], x.shape[1], False, True)
    return (x.new_empty((x.shape[0], w.shape[0])), q_col, s_col, *_weight_fake(w, w.shape[1], w.shape[0]))


@torch.library.custom_op(f"{_LIB}::linear_fp8_backward", mutates_args=())
def linear_fp8_backward(dy: Tensor, xq: Tensor, xs: Tensor, wq: Tensor, ws: Tensor, need_dx: bool = True,
                        need_dw: bool = True, bias: bool = False) -> Tuple[Tensor, Tensor, Tensor]:
    dx, dw, db = dy.new_empty((0,)), dy.new_empty((0,)), dy.new_empty((0,))
    if need_dx or need_dw:
        q_row, q_col, s_row, s_col = _quant_fp8(dy, rowwise=need_dx, colwise=need_dw)
        if need_dx:
            dx = _product_fp8(q_row, s_row, wq, ws)
        if need_dw:
            dw = _product_fp8(q_col, s_col, xq, xs, w_scales="row")
    if bias:   # the column sums alone, of a product without terms
        db = _linear_bwd(dy, dy.new_empty((dy.shape[0], 0)), dy.new_empty((dy.shape[1], 0)), bias=True, need_dx=False,
                         need_dw=False)[2]
    return dx, dw, db


@linear_fp8_backward.register_fake
def _(dy, xq, xs, wq, ws, need_dx=True, need_dw=True, bias=False):
    return (dy.new_empty((dy.shape[0], wq.shape[0]) if need_dx else (0,)),
            dy.new_empty((dy.shape[1], xq.shape[0]) if need_dw else (0,)),
            dy.new_empty((dy.shape[1],) if bias else (0,)))


def _fp8_setup(ctx, inputs, output):
    if ctx.needs_input_grad[1] and inputs[0].shape[0] > _MAX_ROW_SUM:
        raise ValueError(f"x must have at most {_MAX_ROW_SUM} rows for the gradient of w, got {inputs[0].shape[0]}")
    ctx.save_for_backward(*output[1:])
    ctx.mark_non_differentiable(*output[1:])


def _fp8_grad(ctx, dy, *_):
    need = (tuple(ctx.needs_input_grad) + (False,) * 4)[:4]
    dy = _incoming(dy)
    grads = linear_fp8_backward(dy, *ctx.saved_tensors, *need[:3])
    return (*(g if n else None for g, n in zip(grads, need)), dy if need[3] else None)


linear_fp8.register_autograd(_fp8_grad, setup_context=_fp8_setup)

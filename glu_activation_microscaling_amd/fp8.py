"""Binding of 8-bit floating point with a scale for each block of 128: quantizers and products.

Argument marshalling only, as for the other entry points (C names and formulas in
include/glu_mx.h); every function is also a name of the package:
  glu_quant_fp8(x, rowwise=, colwise=)                    -> (q_row, q_col, s_row, s_col)
  glu_fwd_fp8(gate, up, act=, layout=, rowwise=, colwise=) -> the same of act(gate) * up
  glu_quant_fp8_weight(w, transpose=)                     -> (q, s, qt, st)
  glu_linear_fp8(xq, xs, wq, ws, bias, residual, ...)     -> y
Codes are uint8 (E4M3), scales float32.  Code rows are filled up with zero codes to a multiple of 16, so
that each is the K of a product.  What is disabled comes back zero-sized (fixed arity).
"""
from . import ACT, LAYOUT, _flags
from .ffn import _BF16, _F32, _I32, _allocator, _launch, _like, _matrix, _ptr, _same_device, _size
from .gated import _U8, _choice, _glu_operands

W_SCALES = {"block": 0, "row": 1}


def _padded(n):
    return (n + 15) // 16 * 16


def _blocks(n):
    return (n + 127) // 128


def _directions(t, M, N, rowwise, colwise):
    new = _allocator(t)

    def pair(on, rows, cols):
        if not on:
            return new((0,), _U8), new((0,), _F32)
        return new((rows, _padded(cols)), _U8), new((_blocks(cols), rows), _F32)
    (q_row, s_row), (q_col, s_col) = pair(rowwise, M, N), pair(colwise, N, M)
    return q_row, q_col, s_row, s_col


def glu_quant_fp8(x, *, rowwise=True, colwise=False):
    """E4M3 codes and scales of BF16 x [M, N]: q_row [M, N up to 16], s_row [ceil(N/128), M], a scale for
    each 128 of a row; q_col [N, M up to 16], s_col [ceil(M/128), N], a scale for each 128 of a
    column: (q_row, q_col, s_row, s_col)."""
    flags = _flags(rowwise, colwise)
    ld = _matrix(x, "x", _BF16)
    M, N = x.shape
    out = _directions(x, M, N, rowwise, colwise)
    q_row, q_col, s_row, s_col = (_ptr(t) for t in out)
    _launch(x, "glu_quant_fp8", flags, M, N, _ptr(x), ld, q_row, s_row, q_col, s_col)
    return out


def glu_fwd_fp8(gate, up=None, *, act="swiglu", layout="split", rowwise=True, colwise=False):
    """glu_quant_fp8 of h = bf16(act(gate) * up) without writing h: (q_row, q_col, s_row, s_col)."""
    a, lay, flags = _choice(act, ACT, "act"), _choice(layout, LAYOUT, "layout"), _flags(rowwise, colwise)
    M, N, ld = _glu_operands(gate, up, layout)
    _same_device(gate, up)
    out = _directions(gate, M, N, rowwise, colwise)
    q_row, q_col, s_row, s_col = (_ptr(t) for t in out)
    _launch(gate, "glu_fwd_fp8", a, lay, flags, M, N, _ptr(gate), _ptr(up), ld, q_row, s_row, q_col, s_col)
    return out


def glu_quant_fp8_weight(w, *, transpose=False):
    """E4M3 codes of BF16 w [N, K] or [groups, N, K] with a scale for each 128 x 128: q [.., N, K up to 16],
    s [.., ceil(N/128), ceil(K/128)], and with transpose those of the transposed matrix, qt [.., K, N up to
    16], st [.., ceil(K/128), ceil(N/128)]: (q, s, qt, st)."""
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [groups, N, K]")
    _like(w, "w", _BF16, w.shape)
    lead, (N, K), new = w.shape[:-2], w.shape[-2:], _allocator(w)

    def pair(on, n, k):
        if not on:
            return new((0,), _U8), new((0,), _F32)
        return new((*lead, n, _padded(k)), _U8), new((*lead, _blocks(n), _blocks(k)), _F32)
    (q, s), (qt, st) = pair(True, N, K), pair(transpose, K, N)
    _launch(w, "glu_quant_fp8_weight", lead[0] if lead else 1, N, K, _ptr(w), _ptr(q), _ptr(s), _ptr(qt), _ptr(st))
    return q, s, qt, st


def glu_linear_fp8(xq, xs, wq, ws, bias=None, residual=None, *, w_scales="block", offsets=None, out=None):
    """y = x W^T + bias + residual, BF16 [M, N], of codes xq [M, K] with scales xs [ceil(K/128), M] and wq
    [N, K] with ws [ceil(N/128), ceil(K/128)] (w_scales "block") or [ceil(K/128), N] ("row": W quantized
    along the sum).  With int32 offsets [groups + 1], wq, ws and bias have a leading [groups], rows
    offsets[e] .. offsets[e + 1] - 1 go through matrix e, and rows of no group give zeros."""
    mode = _choice(w_scales, W_SCALES, "w_scales")
    if wq.dim() not in (2, 3):
        raise ValueError("wq must be [N, K], or [groups, N, K] with offsets")
    if (wq.dim() == 3) != (offsets is not None):
        raise ValueError("offsets go with wq [groups, N, K], and only with it")
    if xq.dim() != 2:
        raise ValueError("xq must be [M, K]")
    lead, (N, K), M = wq.shape[:-2], wq.shape[-2:], xq.shape[0]
    groups, kb = lead[0] if lead else 1, _blocks(K)
    _like(xq, "xq", _U8, (M, K))
    _like(xs, "xs", _F32, (kb, M))
    _like(wq, "wq", _U8, wq.shape)
    _like(ws, "ws", _F32, (*lead, *((_blocks(N), kb) if mode == 0 else (kb, N))))
    if bias is not None:
        _like(bias, "bias", _BF16, (*lead, N))
    if offsets is not None:
        _like(offsets, "offsets", _I32, (groups + 1,))
    _same_device(xq, xs, wq, ws, bias, residual, offsets, out)
    ld_res = 0 if residual is None else _matrix(residual, "residual", _BF16, M, N)
    new = _allocator(xq)
    if out is None:
        y, ld_y = new((M, N), _BF16), N
    else:
        y, ld_y = out, _matrix(out, "out", _BF16, M, N)
    nbytes = _size("glu_linear_fp8_work_bytes", M, N, K, groups, int(offsets is not None))
    work = new((nbytes,), _U8) if nbytes > 0 else None
    _launch(xq, "glu_linear_fp8", mode, M, N, K, groups, _ptr(offsets), _ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(bias),
            _ptr(residual), ld_res, _ptr(y), ld_y, _ptr(work), nbytes)
    return y

"""Refusals of the gated projections, the checkpoints and the 8-bit products (no GPU): the glu_check_*
exports run the entry points' checks on fake, never-dereferenced pointers, and sizes of scratch
memory are defined for every extent."""
import ctypes
import itertools
import os

import pytest
import torch

import glu_activation_microscaling_amd as glu
from glu_activation_microscaling_amd import ffn
from test_abi_host import ALIGN, ARG, NULL, OK, OVERLAP, SHAPE, STRIDE

L = None
A = [(i + 1) << 34 for i in range(20)]   # fake 16-byte aligned device addresses, 16 GiB apart


def setup_module(module):
    global L
    if not os.path.exists(glu.LIB_PATH):
        from glu_activation_microscaling_amd import build
        build.build()
    L = glu.lib()


def P(addr):
    return ctypes.c_void_p(addr or None)


def call(fn, order, ptrs, base, kw):
    a = dict(base)
    a.update(kw)
    return getattr(L, fn)(*(P(a[k]) if k in ptrs else a[k] for k in order.split()))


def gated(**kw):
    return call("glu_check_gated_linear", "act lay save M N K groups off x ld_x w bias h ld_h pre extra work bytes",
                {"off", "x", "w", "bias", "h", "pre", "extra", "work"},
                dict(act=0, lay=0, save=2, M=64, N=128, K=256, groups=1, off=0, x=A[0], ld_x=256, w=A[1], bias=A[2], h=A[3],
                     ld_h=128, pre=A[4], extra=A[5], work=A[6], bytes=1 << 30), kw)


def test_gated_linear_checks():
    assert gated() == OK and gated(act=3, lay=1) == OK and gated(bias=0) == OK and gated(save=1) == OK
    assert gated(save=0, pre=0, extra=0) == OK
    assert gated(act=4) == ARG and gated(act=-1) == ARG and gated(lay=2) == ARG and gated(save=3) == ARG
    assert gated(M=-1) == SHAPE and gated(N=100) == SHAPE and gated(K=252) == SHAPE and gated(groups=0) == SHAPE
    assert gated(N=(1 << 19) + 8) == SHAPE and gated(M=1 << 31) == SHAPE and gated(groups=1025, off=A[7]) == SHAPE
    assert gated(K=(1 << 20) + 8) == SHAPE
    assert gated(groups=4) == NULL and gated(groups=4, off=A[7]) == OK and gated(off=A[7] + 2, groups=4) == ALIGN
    assert gated(M=0, x=0, h=0, pre=0) == OK and gated(N=0, w=0, h=0) == OK and gated(K=0, x=0, w=0, ld_x=0) == OK
    assert gated(x=0) == NULL and gated(w=0) == NULL and gated(h=0) == NULL
    assert gated(pre=0) == NULL and gated(extra=0) == NULL and gated(save=1, extra=0) == NULL
    assert gated(save=0) == ARG and gated(save=0, pre=0) == ARG
    assert gated(ld_x=248) == STRIDE and gated(ld_x=260) == STRIDE and gated(ld_h=132) == STRIDE
    assert gated(ld_x=(1 << 21) + 8) == STRIDE
    assert gated(x=A[0] + 2) == ALIGN and gated(bias=A[2] + 8) == ALIGN and gated(pre=A[4] + 4) == ALIGN
    assert gated(extra=A[5] + 8) == ALIGN
    assert gated(h=A[0]) == OVERLAP and gated(pre=A[3]) == OVERLAP and gated(extra=A[4]) == OVERLAP
    assert gated(h=A[1] + 256 * 512 - 128) == OVERLAP      # the last rows of w: there are 2 N of them
    assert gated(pre=A[0], M=1) == OVERLAP and gated(h=A[2]) == OVERLAP and gated(off=A[3], groups=4) == OVERLAP
    big = dict(M=300, K=4096, ld_x=4096, N=64, ld_h=64)
    need = L.glu_gated_linear_work_bytes(2, 300, 64, 4096, 1, 0)
    assert need > 0
    assert gated(**big, bytes=need) == OK and gated(**big, bytes=need - 1) == SHAPE
    assert gated(**big, work=0, bytes=0) == NULL and gated(**big, work=A[4], bytes=need) == OVERLAP


def gated_bwd(**kw):
    return call("glu_check_gated_linear_bwd",
                "act lay save M N K groups off dh ld_dh x ld_x w pre extra dx ld_dx dw db h ld_h work bytes",
                {"off", "dh", "x", "w", "pre", "extra", "dx", "dw", "db", "h", "work"},
                dict(act=0, lay=0, save=2, M=64, N=128, K=256, groups=1, off=0, dh=A[0], ld_dh=128, x=A[1], ld_x=256, w=A[2],
                     pre=A[3], extra=A[4], dx=A[5], ld_dx=256, dw=A[6], db=A[7], h=A[8], ld_h=128, work=A[9],
                     bytes=1 << 30), kw)


def test_gated_linear_bwd_checks():
    assert gated_bwd() == OK and gated_bwd(save=1) == OK and gated_bwd(save=1, extra=0) == OK
    assert gated_bwd(save=0) == ARG and gated_bwd(act=9) == ARG and gated_bwd(extra=0) == NULL and gated_bwd(pre=0) == NULL
    assert gated_bwd(dx=0, w=0) == OK and gated_bwd(dw=0, x=0) == OK and gated_bwd(db=0) == OK and gated_bwd(h=0) == OK
    assert gated_bwd(x=0) == NULL and gated_bwd(w=0) == NULL and gated_bwd(dh=0) == NULL
    assert gated_bwd(N=4) == SHAPE and gated_bwd(groups=2) == NULL and gated_bwd(groups=2, off=A[10]) == OK
    assert gated_bwd(ld_dx=128) == STRIDE and gated_bwd(ld_dh=129) == STRIDE and gated_bwd(ld_h=120) == STRIDE
    assert gated_bwd(dw=A[6] + 2) == ALIGN and gated_bwd(db=A[7] + 8) == ALIGN and gated_bwd(work=A[9] + 4) == ALIGN
    assert gated_bwd(dx=A[0]) == OVERLAP and gated_bwd(db=A[6]) == OVERLAP and gated_bwd(h=A[3]) == OVERLAP
    assert gated_bwd(dw=A[2]) == OVERLAP and gated_bwd(work=A[8]) == OVERLAP
    need = L.glu_gated_linear_bwd_work_bytes(64, 128, 256, 1, 0, 1)
    assert need >= 4 * 64 * 128
    assert gated_bwd(bytes=need) == OK and gated_bwd(bytes=need - 1) == SHAPE and gated_bwd(work=0, bytes=0) == NULL
    assert gated_bwd(M=0, dh=0, x=0, pre=0, extra=0, dx=0, h=0) == OK


def fwd_ckpt(**kw):
    return call("glu_check_fwd_ckpt", "act lay M N gate up ld h ld_h q s", {"gate", "up", "h", "q", "s"},
                dict(act=0, lay=0, M=64, N=72, gate=A[0], up=A[1], ld=72, h=A[2], ld_h=72, q=A[3], s=A[4]), kw)


def bwd_ckpt(**kw):
    return call("glu_check_bwd_ckpt", "act lay M N q s dh ld_dh d ld_d h ld_h", {"q", "s", "dh", "d", "h"},
                dict(act=0, lay=0, M=64, N=72, q=A[0], s=A[1], dh=A[2], ld_dh=72, d=A[3], ld_d=144, h=A[4], ld_h=72), kw)


def test_ckpt_checks():
    assert fwd_ckpt() == OK and fwd_ckpt(h=0, ld_h=0) == OK and fwd_ckpt(lay=1, up=0, ld=144) == OK
    assert fwd_ckpt(act=4) == ARG and fwd_ckpt(lay=2) == ARG and fwd_ckpt(lay=1, ld=144) == ARG
    assert fwd_ckpt(N=71) == SHAPE and fwd_ckpt(M=-1) == SHAPE and fwd_ckpt(N=(1 << 28) + 8, ld=1 << 30) == SHAPE
    assert fwd_ckpt(gate=0) == NULL and fwd_ckpt(up=0) == NULL and fwd_ckpt(q=0) == NULL and fwd_ckpt(s=0) == NULL
    assert fwd_ckpt(ld=64) == STRIDE and fwd_ckpt(ld=76) == STRIDE and fwd_ckpt(ld_h=64) == STRIDE
    assert fwd_ckpt(lay=1, up=0, ld=72) == STRIDE
    assert fwd_ckpt(q=A[3] + 8) == ALIGN and fwd_ckpt(up=A[1] + 2) == ALIGN and fwd_ckpt(s=A[4] + 4) == ALIGN
    assert fwd_ckpt(h=A[0]) == OVERLAP and fwd_ckpt(s=A[3] + 144) == OVERLAP and fwd_ckpt(q=A[1]) == OVERLAP
    assert fwd_ckpt(M=0, gate=0, q=0) == OK and fwd_ckpt(N=0, gate=0) == OK
    assert bwd_ckpt() == OK and bwd_ckpt(h=0) == OK and bwd_ckpt(lay=1) == OK
    assert bwd_ckpt(q=0) == NULL and bwd_ckpt(d=0) == NULL and bwd_ckpt(dh=0) == NULL and bwd_ckpt(act=-1) == ARG
    assert bwd_ckpt(ld_d=136) == STRIDE and bwd_ckpt(ld_dh=64) == STRIDE and bwd_ckpt(ld_h=76) == STRIDE
    assert bwd_ckpt(d=A[2]) == OVERLAP and bwd_ckpt(h=A[3] + 128) == OVERLAP and bwd_ckpt(d=A[0]) == OVERLAP
    assert bwd_ckpt(d=A[3] + 4) == ALIGN
    assert L.glu_ckpt_scale_bytes(10, 72) == 60 and L.glu_ckpt_scale_bytes(10, 64) == 40
    assert L.glu_ckpt_scale_bytes(10, 3) == -1 and L.glu_ckpt_scale_bytes(-1, 8) == -1


def quant(**kw):
    return call("glu_check_quant_fp8", "flags M N x ld q_row s_row q_col s_col", {"x", "q_row", "s_row", "q_col", "s_col"},
                dict(flags=3, M=64, N=136, x=A[0], ld=136, q_row=A[1], s_row=A[2], q_col=A[3], s_col=A[4]), kw)


def glu_fp8(**kw):
    return call("glu_check_fwd_fp8", "act lay flags M N gate up ld q_row s_row q_col s_col",
                {"gate", "up", "q_row", "s_row", "q_col", "s_col"},
                dict(act=0, lay=0, flags=1, M=64, N=136, gate=A[0], up=A[5], ld=136, q_row=A[1], s_row=A[2], q_col=0,
                     s_col=0), kw)


def weight(**kw):
    return call("glu_check_quant_fp8_weight", "groups N K w q s qt st", {"w", "q", "s", "qt", "st"},
                dict(groups=2, N=136, K=264, w=A[0], q=A[1], s=A[2], qt=A[3], st=A[4]), kw)


def test_quantizer_checks():
    assert quant() == OK and quant(flags=1, q_col=0, s_col=0) == OK and quant(flags=2, q_row=0, s_row=0) == OK
    assert quant(flags=0) == ARG and quant(flags=4) == ARG and quant(flags=1) == ARG and quant(flags=2) == ARG
    assert quant(q_col=0) == NULL and quant(s_row=0) == NULL and quant(x=0) == NULL
    assert quant(N=132) == SHAPE and quant(M=-1) == SHAPE and quant(ld=128) == STRIDE and quant(ld=140) == STRIDE
    assert quant(x=A[0] + 8) == ALIGN and quant(s_col=A[4] + 4) == ALIGN
    assert quant(q_row=A[0]) == OVERLAP and quant(s_row=A[1] + 144 * 64 - 16) == OVERLAP     # rows of 144 codes
    assert quant(s_row=A[1] + 144 * 64) == OK and quant(M=0, x=0, q_row=0) == OK
    assert glu_fp8() == OK and glu_fp8(act=4) == ARG and glu_fp8(lay=3) == ARG and glu_fp8(up=0) == NULL
    assert glu_fp8(lay=1) == ARG and glu_fp8(lay=1, up=0, ld=272) == OK and glu_fp8(lay=1, up=0) == STRIDE
    assert weight() == OK and weight(qt=0, st=0) == OK and weight(qt=0) == NULL and weight(st=0) == NULL
    assert weight(N=130) == SHAPE and weight(K=260) == SHAPE and weight(groups=-1) == SHAPE and weight(groups=1025) == SHAPE
    assert weight(w=0) == NULL and weight(q=A[1] + 8) == ALIGN and weight(qt=A[1]) == OVERLAP and weight(s=A[0]) == OVERLAP
    assert weight(groups=0, w=0) == OK and weight(N=0, w=0) == OK


def product(**kw):
    return call("glu_check_linear_fp8", "mode M N K groups off xq xs wq ws bias res ld_res y ld_y work bytes",
                {"off", "xq", "xs", "wq", "ws", "bias", "res", "y", "work"},
                dict(mode=0, M=64, N=136, K=272, groups=1, off=0, xq=A[0], xs=A[1], wq=A[2], ws=A[3], bias=A[4], res=A[5],
                     ld_res=136, y=A[6], ld_y=136, work=A[7], bytes=1 << 30), kw)


def test_product_checks():
    assert product() == OK and product(mode=1) == OK and product(bias=0, res=0) == OK and product(mode=2) == ARG
    assert product(M=-1) == SHAPE and product(N=132) == SHAPE and product(K=264) == SHAPE and product(groups=0) == SHAPE
    assert product(K=(1 << 20) + 16) == SHAPE and product(N=(1 << 20) + 8) == SHAPE and product(M=1 << 31) == SHAPE
    assert product(groups=4) == NULL and product(groups=4, off=A[8]) == OK and product(groups=4, off=A[8] + 1) == ALIGN
    assert product(xq=0) == NULL and product(xs=0) == NULL and product(ws=0) == NULL and product(y=0) == NULL
    assert product(K=0, xq=0, xs=0, wq=0, ws=0) == OK and product(M=0, xq=0, y=0) == OK and product(N=0, y=0) == OK
    assert product(ld_y=128) == STRIDE and product(ld_res=140) == STRIDE and product(ld_y=(1 << 21) + 8) == STRIDE
    assert product(xs=A[1] + 4) == ALIGN and product(wq=A[2] + 8) == ALIGN and product(y=A[6] + 2) == ALIGN
    assert product(y=A[0]) == OVERLAP and product(y=A[5]) == OVERLAP and product(y=A[3]) == OVERLAP
    # a scale for each row of W and block takes more than one for each 128 x 128
    assert product(y=A[3] + 64) == OK and product(y=A[3] + 64, mode=1) == OVERLAP
    big = dict(M=300, N=264, K=16384, ld_y=264, ld_res=264)
    need = L.glu_linear_fp8_work_bytes(300, 264, 16384, 1, 0)
    assert need > 0
    assert product(**big, bytes=need) == OK and product(**big, bytes=need - 1) == SHAPE
    assert product(**big, work=0, bytes=0) == NULL and product(**big, work=A[6], bytes=need) == OVERLAP


def test_scratch_sizes_are_defined():
    rows, widths, sums = (0, 1, 8, 9, 33, 129, 1000, 16384, 1 << 20), (0, 8, 72, 1000, 16384), (0, 16, 1008, 65536)
    for M, N, K in itertools.product(rows, widths, sums):
        for groups, grouped in ((1, 0), (1, 1), (64, 1)):
            for save in range(3):
                assert L.glu_gated_linear_work_bytes(save, M, N, K, groups, grouped) >= 0
            assert L.glu_gated_linear_bwd_work_bytes(M, N, K, groups, grouped, 1) >= 4 * M * N
            assert L.glu_linear_fp8_work_bytes(M, N, K, groups, grouped) >= 0
    assert L.glu_gated_linear_work_bytes(3, 8, 8, 8, 1, 0) == -1 and L.glu_gated_linear_work_bytes(0, 8, 9, 8, 1, 0) == -1
    assert L.glu_gated_linear_bwd_work_bytes(8, 8, 8, 2, 0, 0) == -1 and L.glu_linear_fp8_work_bytes(8, 8, 8, 1, 0) == -1


def test_binding_refuses_before_the_call():
    b = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype)   # CPU tensors  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        glu.glu_gated_linear(b(4, 16), b(32, 16))
    with pytest.raises(ValueError, match="act"):
        glu.glu_gated_linear(b(4, 16), b(32, 16), act="silu")
    with pytest.raises(ValueError, match="w_layout"):
        glu.glu_gated_linear(b(4, 16), b(32, 16), w_layout="both")
    with pytest.raises(ValueError, match="w must be"):
        glu.glu_gated_linear(b(4, 16), b(33, 16))
    with pytest.raises(ValueError, match="offsets"):
        glu.glu_gated_linear(b(4, 16), b(2, 32, 16))
    with pytest.raises(ValueError, match="GPU"):
        glu.glu_fwd_ckpt(b(4, 16), b(4, 16))
    with pytest.raises(ValueError, match="layout"):
        glu.glu_fwd_ckpt(b(4, 16), b(4, 16), layout="rows")
    with pytest.raises(ValueError, match="enable"):
        glu.glu_quant_fp8(b(4, 16), rowwise=False)
    with pytest.raises(TypeError):
        glu.glu_quant_fp8(b(4, 16, dtype=torch.float32))
    with pytest.raises(ValueError, match="w must be"):
        glu.glu_quant_fp8_weight(b(4))
    u8, f = dict(dtype=torch.uint8), dict(dtype=torch.float32)
    with pytest.raises(ValueError, match="w_scales"):
        glu.glu_linear_fp8(b(4, 16, **u8), b(1, 4, **f), b(8, 16, **u8), b(1, 1, **f), w_scales="tile")
    with pytest.raises(ValueError, match="offsets"):
        glu.glu_linear_fp8(b(4, 16, **u8), b(1, 4, **f), b(2, 8, 16, **u8), b(2, 1, 1, **f))


def test_the_call_is_made_on_its_operands_device(monkeypatch):
    """With another device current, the call and the stream are those of the operands' device."""
    log = []

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            log.append(("enter", self.i))

        def __exit__(self, *_):
            log.append(("exit", self.i))

    class Operand:
        def get_device(self):
            return 3

    monkeypatch.setattr(ffn, "_device", lambda: 0)
    monkeypatch.setattr(ffn, "_raw_stream", lambda i: ("stream", i))
    monkeypatch.setattr(ffn, "_call", lambda name, *args: log.append((name, args)))
    monkeypatch.setattr(torch.cuda, "device", Device)
    ffn._launch(Operand(), "f", 1, 2)
    assert log == [("enter", 3), ("f", (1, 2, ("stream", 3))), ("exit", 3)]
    log.clear()
    monkeypatch.setattr(ffn, "_device", lambda: 3)
    ffn._launch(Operand(), "f", 1, 2)
    assert log == [("f", (1, 2, ("stream", 3)))]


def test_outputs_are_made_contiguous_and_on_their_operands_device(monkeypatch):
    monkeypatch.setattr(ffn, "_strided", lambda *args: args)
    for shape in ((0,), (5,), (0, 7), (7, 0), (3, 8), (2, 0, 4), (2, 3, 4), (0, 3, 0)):
        for s in (shape, torch.Size(shape)):
            got = ffn._contiguous(s, torch.uint8)
            assert got == (shape, torch.empty(shape).stride(), torch.uint8) and type(got[0]) is type(got[1]) is tuple

    class Operand:
        def get_device(self):
            return 3

        def new_empty(self, shape, dtype):
            return "its own", shape, dtype

    monkeypatch.setattr(ffn, "_device", lambda: 3)
    assert ffn._allocator(Operand()) is ffn._contiguous
    monkeypatch.setattr(ffn, "_device", lambda: 0)
    assert ffn._allocator(Operand())((4, 8), torch.uint8) == ("its own", (4, 8), torch.uint8)
    monkeypatch.setattr(ffn, "_device", lambda: 3)
    monkeypatch.setattr(ffn, "_strided", None)
    assert ffn._allocator(Operand())((4, 8), torch.uint8) == ("its own", (4, 8), torch.uint8)

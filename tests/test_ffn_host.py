"""Refusals of the operators around the GLU (no GPU): the glu_check_* exports run the entry
points' checks on fake, never-dereferenced pointers, and the sizes of scratch memory are defined
for every extent."""
import ctypes
import itertools
import os

import pytest
import torch

import glu_activation_microscaling_amd as glu
from test_abi_host import ALIGN, ARG, NULL, OK, OVERLAP, SHAPE, STRIDE

L = None
# fake 16-byte aligned device addresses, 16 GiB apart
A = [(i + 1) << 34 for i in range(20)]


def setup_module(module):
    global L
    if not os.path.exists(glu.LIB_PATH):
        from glu_activation_microscaling_amd import build
        build.build()
    L = glu.lib()


def P(addr):
    return ctypes.c_void_p(addr or None)


PRE, POST, F32_STREAM, F32_PARAMS, GG, WG, BG = 1, 2, 4, 8, 16, 32, 64


def norm(mx=False, **kw):
    a = dict(kind=0, flags=PRE | POST, M=64, H=128, groups=1, x=A[0], ld_x=128, y=A[1], ld_y=128, gate=A[2],
             w_pre=A[3], b_pre=A[4], w_post=A[5], rs=1.0, eps=1e-6, xo=A[6], ld_xo=128, h=A[7], ld_h=128, q=A[8],
             s=A[9], stats=A[10])
    a.update(kw)
    head = [a["kind"], a["flags"], a["M"], a["H"], a["groups"], P(a["x"]), a["ld_x"], P(a["y"]), a["ld_y"], P(a["gate"]),
            P(a["w_pre"]), P(a["b_pre"]), P(a["w_post"]), a["rs"], a["eps"], P(a["xo"]), a["ld_xo"]]
    if mx:
        return L.glu_check_block_norm_mxfp8(*head, P(a["q"]), P(a["s"]), P(a["stats"]))
    return L.glu_check_block_norm(*head, P(a["h"]), a["ld_h"], P(a["stats"]))


def test_block_norm_checks():
    assert norm() == OK and norm(kind=1) == OK and norm(M=1) == OK
    assert norm(kind=2) == ARG and norm(flags=128 | PRE) == ARG and norm(eps=-1.0) == ARG
    assert norm(eps=float("nan")) == ARG
    assert norm(M=-1) == SHAPE and norm(H=-1) == SHAPE and norm(M=1 << 31) == SHAPE
    assert norm(H=16385, ld_x=16392, ld_y=16392, ld_xo=16392, ld_h=16392) == SHAPE
    assert norm(groups=0) == SHAPE and norm(groups=3) == SHAPE and norm(groups=64) == OK
    assert norm(M=0, x=0, y=0) == OK and norm(H=0, x=0) == OK
    assert norm(x=0) == NULL and norm(xo=0) == NULL and norm(h=0) == NULL and norm(stats=0) == NULL
    assert norm(ld_x=127) == STRIDE and norm(ld_y=127) == STRIDE and norm(ld_xo=120) == STRIDE
    assert norm(ld_h=1) == STRIDE and norm(ld_x=131) == OK
    assert norm(x=A[0] + 2) == ALIGN and norm(gate=A[2] + 8) == ALIGN and norm(stats=A[10] + 4) == ALIGN
    assert norm(flags=PRE) == ARG                       # w_post without the norm after the block
    assert norm(flags=PRE, w_post=0) == OK
    assert norm(flags=POST) == ARG and norm(flags=POST, w_pre=0, b_pre=0) == ARG      # h without its norm
    assert norm(flags=POST, w_pre=0, b_pre=0, h=0) == OK
    assert norm(y=0) == ARG and norm(y=0, gate=0, w_post=0, flags=PRE, xo=0) == OK
    assert norm(y=0, gate=0, w_post=0, flags=PRE) == ARG                              # x_out without y
    assert norm(xo=A[0]) == OVERLAP and norm(h=A[6]) == OVERLAP and norm(h=A[1] + 256 * 63) == OVERLAP
    assert norm(gate=A[6]) == OVERLAP
    # FP32 stream and parameters: twice the bytes, so these now meet
    assert norm(xo=A[0] + 64 * 256) == OK and norm(xo=A[0] + 64 * 256, flags=PRE | POST | F32_STREAM) == OVERLAP
    assert norm(h=A[3] + 256) == OK and norm(h=A[3] + 256, flags=PRE | POST | F32_PARAMS) == OVERLAP
    assert norm(h=A[3] + 256, groups=2, flags=PRE | POST | WG) == OVERLAP
    assert norm(ld_x=1 << 60) == SHAPE


def test_block_norm_mxfp8_checks():
    assert norm(mx=True) == OK
    assert norm(mx=True, H=72, ld_x=128) == SHAPE and norm(mx=True, q=0) == NULL and norm(mx=True, s=0) == NULL
    assert norm(mx=True, ld_x=132) == STRIDE and norm(mx=True, ld_xo=130) == STRIDE
    assert norm(mx=True, flags=POST, w_pre=0, b_pre=0) == ARG
    assert norm(mx=True, s=A[8] + 16) == OVERLAP and norm(mx=True, q=A[8] + 8) == ALIGN


def norm_bwd(**kw):
    a = dict(kind=0, flags=PRE | POST, M=64, H=128, groups=1, x=A[0], ld_x=128, y=A[1], ld_y=128, stats=A[2], dxo=A[3],
             ld_dxo=128, dh=A[4], ld_dh=128, gate=A[5], w_pre=A[6], w_post=A[7], rs=1.0, dx=A[8], ld_dx=128, dy=A[9],
             ld_dy=128, dgate=A[10], dw_pre=A[11], db_pre=A[12], dw_post=A[13], work=A[14], bytes=1 << 30)
    a.update(kw)
    return L.glu_check_block_norm_bwd(a["kind"], a["flags"], a["M"], a["H"], a["groups"], P(a["x"]), a["ld_x"],
                                      P(a["y"]), a["ld_y"], P(a["stats"]), P(a["dxo"]), a["ld_dxo"], P(a["dh"]),
                                      a["ld_dh"], P(a["gate"]), P(a["w_pre"]), P(a["w_post"]), a["rs"], P(a["dx"]),
                                      a["ld_dx"], P(a["dy"]), a["ld_dy"], P(a["dgate"]), P(a["dw_pre"]), P(a["db_pre"]),
                                      P(a["dw_post"]), P(a["work"]), a["bytes"])


def test_block_norm_bwd_checks():
    assert norm_bwd() == OK and norm_bwd(dxo=0) == OK
    assert norm_bwd(dgate=0, dw_pre=0, db_pre=0, dw_post=0, work=0, bytes=0) == OK
    assert norm_bwd(work=0) == NULL and norm_bwd(bytes=16) == SHAPE
    assert norm_bwd(x=0) == NULL and norm_bwd(stats=0) == NULL and norm_bwd(dx=0) == NULL and norm_bwd(dy=0) == NULL
    assert norm_bwd(dh=0) == NULL and norm_bwd(flags=POST, w_pre=0, dw_pre=0, db_pre=0) == ARG   # dh without h
    assert norm_bwd(flags=POST, w_pre=0, dw_pre=0, db_pre=0, dh=0) == OK
    assert norm_bwd(flags=POST, w_pre=0, dw_pre=0, db_pre=0, dh=0, dxo=0) == NULL
    assert norm_bwd(flags=PRE, w_post=0) == ARG and norm_bwd(flags=PRE, w_post=0, dw_post=0) == OK
    assert norm_bwd(y=0, gate=0, w_post=0, flags=PRE, dw_post=0) == ARG                          # dy without y
    assert norm_bwd(y=0, gate=0, w_post=0, flags=PRE, dw_post=0, dy=0, dgate=0) == OK
    assert norm_bwd(ld_dx=100) == STRIDE and norm_bwd(ld_dy=1) == STRIDE and norm_bwd(ld_dh=127) == STRIDE
    assert norm_bwd(dx=A[8] + 2) == ALIGN and norm_bwd(work=A[14] + 4) == ALIGN
    assert norm_bwd(dx=A[3]) == OVERLAP and norm_bwd(dgate=A[10], dw_pre=A[10]) == OVERLAP
    assert norm_bwd(work=A[9]) == OVERLAP
    assert norm_bwd(M=0, x=0, dx=0, work=0, bytes=0) == OK and norm_bwd(M=0, dgate=A[11]) == OVERLAP
    assert norm_bwd(M=1, bytes=L.glu_block_norm_bwd_work_bytes(1, 128, 1)) == OK


def linear(**kw):
    a = dict(act=0, M=64, N=128, K=256, groups=1, off=0, x=A[0], ld_x=256, w=A[1], bias=A[2], res=A[3], ld_res=128,
             y=A[4], ld_y=128, pre=A[5], work=A[6], bytes=1 << 30)
    a.update(kw)
    return L.glu_check_linear(a["act"], a["M"], a["N"], a["K"], a["groups"], P(a["off"]), P(a["x"]), a["ld_x"],
                              P(a["w"]), P(a["bias"]), P(a["res"]), a["ld_res"], P(a["y"]), a["ld_y"], P(a["pre"]),
                              P(a["work"]), a["bytes"])


def test_linear_checks():
    assert linear() == OK and linear(bias=0, res=0, pre=0) == OK
    assert linear(act=4) == ARG and linear(act=-1) == ARG
    assert linear(M=-1) == SHAPE and linear(N=100) == SHAPE and linear(K=252) == SHAPE and linear(groups=0) == SHAPE
    assert linear(N=(1 << 20) + 8) == SHAPE and linear(M=1 << 31) == SHAPE and linear(groups=1025, off=A[7]) == SHAPE
    assert linear(groups=4) == NULL and linear(groups=4, off=A[7]) == OK and linear(off=A[7] + 2, groups=4) == ALIGN
    assert linear(M=0, x=0, y=0) == OK and linear(K=0, x=0, w=0, ld_x=0) == OK
    assert linear(x=0) == NULL and linear(w=0) == NULL and linear(y=0) == NULL
    assert linear(ld_x=248) == STRIDE and linear(ld_x=260) == STRIDE and linear(ld_y=132) == STRIDE
    assert linear(ld_res=120) == STRIDE and linear(ld_x=(1 << 21) + 8) == STRIDE
    assert linear(x=A[0] + 2) == ALIGN and linear(bias=A[2] + 8) == ALIGN and linear(pre=A[5] + 4) == ALIGN
    assert linear(y=A[0]) == OVERLAP and linear(pre=A[4]) == OVERLAP and linear(y=A[3]) == OVERLAP
    # 300 rows of 128 columns and a long sum: split, so scratch memory is needed
    need = L.glu_linear_work_bytes(300, 128, 4096, 1, 0)
    assert need > 0
    big = dict(M=300, K=4096, ld_x=4096)
    assert linear(**big, bytes=need) == OK and linear(**big, bytes=need - 1) == SHAPE
    assert linear(**big, work=0, bytes=0) == NULL and linear(**big, work=A[4], bytes=need) == OVERLAP


def linear_bwd(**kw):
    a = dict(act=1, M=64, N=128, K=256, groups=1, off=0, dy=A[0], ld_dy=128, x=A[1], ld_x=256, w=A[2], pre=A[3],
             dx=A[4], ld_dx=256, dw=A[5], db=A[6], work=A[7], bytes=1 << 30)
    a.update(kw)
    return L.glu_check_linear_bwd(a["act"], a["M"], a["N"], a["K"], a["groups"], P(a["off"]), P(a["dy"]), a["ld_dy"],
                                  P(a["x"]), a["ld_x"], P(a["w"]), P(a["pre"]), P(a["dx"]), a["ld_dx"], P(a["dw"]),
                                  P(a["db"]), P(a["work"]), a["bytes"])


def test_linear_bwd_checks():
    assert linear_bwd() == OK and linear_bwd(act=0, pre=0) == OK
    assert linear_bwd(pre=0) == NULL and linear_bwd(act=0) == ARG and linear_bwd(act=9) == ARG
    assert linear_bwd(dx=0, w=0) == OK and linear_bwd(dw=0, x=0) == OK and linear_bwd(db=0) == OK
    assert linear_bwd(x=0) == NULL and linear_bwd(w=0) == NULL and linear_bwd(dy=0) == NULL
    assert linear_bwd(N=4) == SHAPE and linear_bwd(groups=2) == NULL and linear_bwd(groups=2, off=A[9]) == OK
    assert linear_bwd(ld_dx=128) == STRIDE and linear_bwd(ld_dy=129) == STRIDE
    assert linear_bwd(dw=A[5] + 2) == ALIGN and linear_bwd(dx=A[0]) == OVERLAP and linear_bwd(db=A[5]) == OVERLAP
    assert linear_bwd(work=0, bytes=0) == NULL and linear_bwd(bytes=64) == SHAPE
    assert linear_bwd(M=0, dy=0, x=0, pre=0, dx=0) == OK


def sort(**kw):
    a = dict(T=100, k=4, E=8, ids=A[0], b=4, rows=A[1], off=A[2], work=A[3], bytes=1 << 20)
    a.update(kw)
    return L.glu_check_moe_sort(a["T"], a["k"], a["E"], P(a["ids"]), a["b"], P(a["rows"]), P(a["off"]), P(a["work"]),
                                a["bytes"])


def test_moe_checks():
    assert sort() == OK and sort(b=8) == OK and sort(b=2) == ARG
    assert sort(T=-1) == SHAPE and sort(E=0) == SHAPE and sort(E=1025) == SHAPE and sort(T=1 << 30) == SHAPE
    assert sort(T=1 << 62, k=4) == SHAPE
    assert sort(ids=0) == NULL and sort(rows=0) == NULL and sort(off=0) == NULL
    assert sort(T=0, ids=0, rows=0) == OK and sort(T=0, off=0) == NULL
    assert sort(ids=A[0] + 4) == ALIGN and sort(rows=A[0]) == OVERLAP and sort(off=A[1]) == OVERLAP
    assert sort(T=5000, bytes=0) == SHAPE and sort(T=5000, work=0, bytes=0) == NULL

    def permute(**kw):
        a = dict(T=100, k=4, E=8, rb=256, x=A[0], ld_x=256, rows=A[1], off=A[2], xs=A[3], ld_xs=256)
        a.update(kw)
        return L.glu_check_moe_permute(a["T"], a["k"], a["E"], a["rb"], P(a["x"]), a["ld_x"], P(a["rows"]), P(a["off"]),
                                       P(a["xs"]), a["ld_xs"])

    assert permute() == OK and permute(rb=33) == OK and permute(rb=0, x=0) == OK and permute(k=0, xs=0) == OK
    assert permute(rb=-1) == SHAPE and permute(rb=(1 << 24) + 1) == SHAPE and permute(x=0) == NULL
    assert permute(ld_x=255) == STRIDE and permute(ld_xs=0) == STRIDE and permute(xs=A[0]) == OVERLAP
    assert permute(off=A[2] + 4) == ALIGN and permute(off=0) == NULL

    def combine(**kw):
        a = dict(T=100, k=4, H=128, y=A[0], ld_y=128, rows=A[1], w=A[2], res=A[3], ld_res=128, out=A[4], ld_out=128)
        a.update(kw)
        return L.glu_check_moe_combine(a["T"], a["k"], a["H"], P(a["y"]), a["ld_y"], P(a["rows"]), P(a["w"]),
                                       P(a["res"]), a["ld_res"], P(a["out"]), a["ld_out"])

    assert combine() == OK and combine(w=0, res=0) == OK and combine(k=0, y=0, rows=0, w=0) == OK
    assert combine(T=0, out=0) == OK and combine(out=0) == NULL and combine(y=0) == NULL
    assert combine(H=-1) == SHAPE and combine(ld_y=100) == STRIDE and combine(ld_out=1) == STRIDE
    assert combine(out=A[3]) == OVERLAP and combine(out=A[0] + 256 * 399) == OVERLAP and combine(w=A[2] + 4) == ALIGN

    def bwd(**kw):
        a = dict(T=100, k=4, H=128, E=8, dout=A[0], ld_dout=128, y=A[1], ld_y=128, rows=A[2], w=A[3], off=A[4], dy=A[5],
                 ld_dy=128, dw=A[6])
        a.update(kw)
        return L.glu_check_moe_combine_bwd(a["T"], a["k"], a["H"], a["E"], P(a["dout"]), a["ld_dout"], P(a["y"]),
                                           a["ld_y"], P(a["rows"]), P(a["w"]), P(a["off"]), P(a["dy"]), a["ld_dy"],
                                           P(a["dw"]))

    assert bwd() == OK and bwd(T=0, rows=0) == OK and bwd(w=0) == NULL and bwd(dw=0) == NULL and bwd(dy=0) == NULL
    assert bwd(dy=A[1]) == OVERLAP and bwd(ld_dy=64) == STRIDE and bwd(E=0) == SHAPE and bwd(dw=A[6] + 8) == ALIGN


def test_scratch_sizes_are_defined_for_every_extent():
    n = [0, 1, 7, 8, 64, 1000, 40000]
    for M, N, K, G, grouped in itertools.product(n, [0, 8, 64, 1000, 7168], [0, 8, 64, 4096], [1, 2, 64], [0, 1]):
        want = -1 if G > 1 and not grouped else 0
        size = L.glu_linear_work_bytes(M, N, K, G, grouped)
        assert size == -1 if want else size >= 0
        for act, bias in itertools.product(range(4), range(2)):
            size = L.glu_linear_bwd_work_bytes(act, M, N, K, G, grouped, bias)
            assert size == -1 if want else size >= (2 * M * N if act else 0)
    for M, H, G in itertools.product(n, [0, 1, 8, 64, 8193, 16384], [1, 2, 8, 64, 5000]):
        size = L.glu_block_norm_bwd_work_bytes(M, H, G)
        assert size == -1 if M % G else size >= 0
    assert L.glu_linear_work_bytes(-1, 8, 8, 1, 0) == L.glu_linear_bwd_work_bytes(7, 8, 8, 8, 1, 0, 0) == -1
    for T, k, E in itertools.product(n, [0, 1, 8], [1, 64, 1024]):
        assert L.glu_moe_sort_work_bytes(T, k, E) >= 0
    assert L.glu_moe_sort_work_bytes(1, 1, 0) == -1


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        glu.glu_block_norm(x)
    with pytest.raises(TypeError):
        glu.glu_block_norm(x.half())
    with pytest.raises(ValueError):
        glu.glu_block_norm(x, kind="batch")
    with pytest.raises(ValueError):
        glu.glu_linear(x, x)
    with pytest.raises(ValueError):
        glu.glu_linear(x, x, act="relu")
    with pytest.raises(ValueError):
        glu.glu_linear(x, x.reshape(1, 4, 64))
    with pytest.raises(TypeError):
        glu.glu_moe_sort(x, 4)
    with pytest.raises(ValueError):
        glu.glu_moe_sort(torch.zeros(4, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        glu.glu_moe_combine(x, torch.zeros(4, 1, dtype=torch.int32))

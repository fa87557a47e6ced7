"""Refusals of the layer calls, before any launch (no kernel runs, so fake
pointer values are safe), and the binding's own checks on the CPU."""
import ctypes

import pytest
import torch

from learnable_scale_fake_gb300 import _build, aqfq

OK, NULL, SHAPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5
A = 0x10000
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    _build.build()
    return aqfq.lib()


def ck(fmt=aqfq.INT8, group=128, codes=7 * A, scale=8 * A):
    return ctypes.byref(aqfq.Ckpt8(fmt, group, codes, scale))


def pack(L, c=None, dtype=0, x=A, ld=64, R=4, C=64):
    return L.aqfq_ckpt8_pack(ck() if c is None else c, dtype, x, ld, R, C, None)


def test_pack_checks(L):
    assert L.aqfq_ckpt8_pack(None, 0, A, 64, 4, 64, None) == NULL
    assert pack(L, ck(fmt=aqfq.INT4)) == UNSUP
    assert pack(L, ck(fmt=aqfq.NVFP4)) == UNSUP
    for g in (0, 16, 48, 256, -128):
        assert pack(L, ck(group=g)) == UNSUP
    assert pack(L, dtype=2) == UNSUP
    assert pack(L, ck(codes=None)) == NULL
    assert pack(L, ck(scale=None)) == NULL
    assert pack(L, ck(scale=A + 2)) == ALIGN
    assert pack(L, x=None) == NULL
    assert pack(L, x=A + 1) == ALIGN
    assert pack(L, dtype=1, x=A + 2) == ALIGN
    assert pack(L, ld=63) == SHAPE
    assert pack(L, R=-1) == SHAPE
    assert pack(L, C=-8) == SHAPE
    assert pack(L, R=1 << 41) == SHAPE
    assert pack(L, C=1 << 33, ld=1 << 33) == SHAPE
    assert pack(L, ck(codes=None, scale=None), x=None, R=0) == OK
    assert pack(L, ck(codes=None, scale=None), x=None, C=0) == OK


def test_unpack_checks(L):
    f = lambda c=None, act=0, dtype=0, y=A, ld=64, R=4, C=64: L.aqfq_ckpt8_unpack(
        ck() if c is None else c, act, dtype, y, ld, R, C, None)
    assert L.aqfq_ckpt8_unpack(None, 0, 0, A, 64, 4, 64, None) == NULL
    assert f(act=5) == UNSUP and f(act=-1) == UNSUP and f(dtype=-1) == UNSUP
    assert f(y=None) == NULL and f(y=A + 1) == ALIGN and f(ld=8) == SHAPE
    assert f(R=0, y=None) == OK


def act_bwd(L, c=None, act=2, dtype=0, dy=A, ldd=64, R=64, C=64, dx=2 * A, ldx=64, y=None, ldy=0,
            db=None, ws=None, wsb=0):
    return L.aqfq_ckpt8_act_bwd(ck() if c is None else c, act, dtype, dy, ldd, R, C, dx, ldx, y, ldy,
                                db, 0, ws, wsb, None)


def test_act_bwd_checks(L):
    none = ctypes.c_void_p(None)
    assert act_bwd(L, none) == NULL                     # an activation needs its checkpoint
    assert act_bwd(L, none, act=0, y=3 * A, ldy=64) == NULL
    assert act_bwd(L, act=9) == UNSUP
    assert act_bwd(L, dtype=3) == UNSUP
    assert act_bwd(L, dy=None) == NULL
    assert act_bwd(L, dx=None) == NULL                  # nothing to compute
    assert act_bwd(L, ldd=60) == SHAPE
    assert act_bwd(L, ldx=60) == SHAPE
    assert act_bwd(L, y=3 * A, ldy=60) == SHAPE
    assert act_bwd(L, dx=A + 1) == ALIGN
    assert act_bwd(L, db=A + 2, ws=A, wsb=1 << 20) == ALIGN
    assert act_bwd(L, db=A) == WS
    need = aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(64, 64)
    assert need == 8 * 64 * 4
    assert act_bwd(L, db=A, ws=A, wsb=need - 1) == WS
    assert act_bwd(L, db=A, ws=A + 4, wsb=need) == ALIGN
    assert act_bwd(L, R=0, dy=None, dx=None) == OK
    assert aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(-1, 64) == 0
    # the scratch is bounded however many rows there are
    assert (aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(10 ** 7, 64)
            == aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(10 ** 8, 64))


def nfwd(L, dtype=0, x=A, ldx=64, R=4, C=64, pd=0, g=A, b=A, eps=1e-5, y=2 * A, ldy=64, m=A, r=A,
         c=None):
    return L.aqfq_layernorm_fwd(dtype, x, ldx, R, C, pd, g, b, ctypes.c_float(eps), y, ldy, m, r, c, None)


def test_layernorm_fwd_checks(L):
    assert nfwd(L, dtype=2) == UNSUP
    assert nfwd(L, pd=-1) == UNSUP
    assert nfwd(L, x=None) == NULL
    assert nfwd(L, y=None) == NULL
    assert nfwd(L, C=0) == SHAPE
    assert nfwd(L, C=-1) == SHAPE
    assert nfwd(L, ldx=32) == SHAPE
    assert nfwd(L, ldy=32) == SHAPE
    assert nfwd(L, eps=-1.0) == SHAPE
    assert nfwd(L, eps=float("nan")) == SHAPE
    assert nfwd(L, eps=float("inf")) == SHAPE
    assert nfwd(L, x=A + 1) == ALIGN
    assert nfwd(L, dtype=1, y=A + 2) == ALIGN
    assert nfwd(L, pd=1, g=A + 2) == ALIGN
    assert nfwd(L, m=A + 1) == ALIGN
    assert nfwd(L, c=ck(group=96)) == UNSUP
    assert nfwd(L, c=ck(codes=None)) == NULL
    assert nfwd(L, R=0, x=None, y=None) == OK


def nbwd(L, dtype=0, dy=A, lddy=64, x=2 * A, ldx=64, c=None, R=64, C=64, m=A, r=A, pd=0, g=A, dres=None,
         lddres=0, dx=3 * A, lddx=64, dg=None, db=None, ws=None, wsb=0):
    return L.aqfq_layernorm_bwd(dtype, dy, lddy, x, ldx, c, R, C, m, r, pd, g, dres, lddres, dx, lddx,
                                dg, db, 0, ws, wsb, None)


def test_layernorm_bwd_checks(L):
    assert nbwd(L, c=ck()) == UNSUP                      # x and its checkpoint
    assert nbwd(L, x=None) == NULL
    assert nbwd(L, dy=None) == NULL
    assert nbwd(L, m=None) == NULL
    assert nbwd(L, r=None) == NULL
    assert nbwd(L, dx=None) == NULL                      # nothing to compute
    assert nbwd(L, dx=None, dg=A, dres=A, lddres=64, ws=A, wsb=1 << 20) == UNSUP
    assert nbwd(L, C=0) == SHAPE
    assert nbwd(L, lddy=63) == SHAPE
    assert nbwd(L, ldx=63) == SHAPE
    assert nbwd(L, lddx=63) == SHAPE
    assert nbwd(L, dres=A, lddres=63) == SHAPE
    assert nbwd(L, dtype=7) == UNSUP
    assert nbwd(L, dy=A + 1) == ALIGN
    assert nbwd(L, dg=A + 2, ws=A, wsb=1 << 20) == ALIGN
    assert nbwd(L, dg=A) == WS
    need = aqfq.aqfq_layernorm_bwd_workspace_bytes(64, 64)
    assert need > 0
    assert nbwd(L, db=A, ws=A, wsb=need - 1) == WS
    assert nbwd(L, db=A, ws=A + 4, wsb=need) == ALIGN
    assert nbwd(L, R=0, dy=None, x=None, m=None, r=None, dx=None) == OK
    assert (aqfq.aqfq_layernorm_bwd_workspace_bytes(10 ** 7, 64)
            == aqfq.aqfq_layernorm_bwd_workspace_bytes(10 ** 8, 64))


def fwd(L, x=A, ldx=64, w=2 * A, ldw=64, M=4, N=32, K=64, bd=0, b=None, act=0, res=None, ldr=0, y=3 * A,
        ldy=32, c=None, ws=None, wsb=0, err=None):
    return L.aqfq_linear_fwd(x, ldx, w, ldw, M, N, K, bd, b, act, res, ldr, y, ldy, c, ws, wsb, err, None)


def dgrad(L, dy=A, lddy=32, w=2 * A, ldw=64, M=4, N=32, K=64, act=0, c=None, res=None, ldr=0, dx=3 * A,
          lddx=64, err=None):
    return L.aqfq_linear_dgrad(dy, lddy, w, ldw, M, N, K, act, c, res, ldr, dx, lddx, None, 0, err, None)


def wgrad(L, dy=A, lddy=32, x=2 * A, ldx=64, M=4, N=32, K=64, dtype=0, dw=3 * A, lddw=64, err=None):
    return L.aqfq_linear_wgrad(dy, lddy, x, ldx, M, N, K, dtype, dw, lddw, 0, None, 0, err, None)


def test_linear_checks(L):
    for f, a, b, o in ((fwd, "x", "w", "y"), (dgrad, "dy", "w", "dx"), (wgrad, "dy", "x", "dw")):
        assert f(L, **{a: None}) == NULL
        assert f(L, **{b: None}) == NULL
        assert f(L, **{o: None}) == NULL
        assert f(L, **{a: A + 8}) == ALIGN
        assert f(L, **{b: A + 2}) == ALIGN
        assert f(L, **{o: A + 1}) == ALIGN
        assert f(L, **{"ld" + a: 68}) == ALIGN           # rows 16-byte aligned
        assert f(L, **{"ld" + b: 68}) == ALIGN
        assert f(L, **{"ld" + a: 24}) == SHAPE
        assert f(L, **{"ld" + b: 56}) == SHAPE
        assert f(L, **{"ld" + o: 24}) == SHAPE
        assert f(L, M=-1) == SHAPE
        assert f(L, N=1 << 30) == SHAPE
        assert f(L, err=A + 2) == ALIGN
    for f in (fwd, dgrad):
        assert f(L, act=5) == UNSUP
        assert f(L, act=-1) == UNSUP
        assert f(L, res=A, ldr=8) == SHAPE
        assert f(L, res=A + 1, ldr=64) == ALIGN
        assert f(L, c=ck(group=16)) == UNSUP
        assert f(L, c=ck(codes=None)) == NULL
    assert dgrad(L, act=1) == NULL                       # a derivative needs its checkpoint
    assert fwd(L, bd=2) == UNSUP
    assert fwd(L, bd=1, b=A + 2) == ALIGN
    assert wgrad(L, dtype=2) == UNSUP
    assert wgrad(L, dtype=1, dw=A + 2) == ALIGN
    # nothing to compute needs no buffers
    assert fwd(L, M=0, x=None, w=None, y=None) == OK
    assert fwd(L, N=0, x=None, w=None, y=None) == OK
    assert dgrad(L, M=0, dy=None, w=None, dx=None) == OK
    assert wgrad(L, K=0, dy=None, x=None, dw=None, ldx=0, lddw=0) == OK
    assert aqfq.aqfq_linear_workspace_bytes(3, 4, 4, 4) == 0
    assert aqfq.aqfq_linear_workspace_bytes(0, -4, 4, 4) == 0


def test_binding_checks_on_the_host():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                      # CPU tensors
        aqfq.aqfq_linear_fwd(t, t, t)
    with pytest.raises(ValueError):
        aqfq.aqfq_layernorm_fwd(t, None, None, 1e-5, t)
    with pytest.raises(ValueError):                      # scale of another shape
        aqfq.ckpt8(aqfq.INT8, 32, torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 3))
    with pytest.raises(TypeError):
        aqfq.ckpt8(aqfq.INT8, 32, t, torch.zeros(4, 2))

"""Refusals of the calls between a layer's quantized products, before any launch (fake
pointer values are safe), the binding's own checks on the CPU, and the host-only calls."""
import ctypes
import math

import pytest
import torch

from learnable_scale_fake_gb300 import _build, aqfq

OK, NULL, SHAPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5
A = 0x10000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return aqfq.lib()


# ---- rotary positions ----------------------------------------------------------------

def hd(x=A, y=2 * A, heads=4, ldx=256, hsx=64, ldy=256, hsy=64):
    return ctypes.byref(aqfq.Heads(x, y, heads, ldx, hsx, ldy, hsy))


def rotary(L, dtype=0, q=None, k=None, T=4, D=64, rot=64, layout=0, pos=3 * A, freqs=4 * A, m=1.0):
    return L.aqfq_rotary(dtype, hd() if q is None else q, k, T, D, rot, layout, pos, freqs, ctypes.c_float(m),
                         0, None)


def test_rotary_checks(L):
    none = ctypes.c_void_p(None)
    assert rotary(L, q=none) == NULL
    assert rotary(L, dtype=2) == UNSUP and rotary(L, layout=2) == UNSUP and rotary(L, layout=-1) == UNSUP
    assert rotary(L, T=-1) == SHAPE
    assert rotary(L, D=0, rot=0) == SHAPE and rotary(L, D=8193) == SHAPE
    assert rotary(L, rot=63) == SHAPE and rotary(L, rot=66) == SHAPE and rotary(L, rot=-2) == SHAPE
    assert rotary(L, pos=None) == NULL and rotary(L, freqs=None) == NULL
    assert rotary(L, pos=A + 4) == ALIGN and rotary(L, freqs=A + 4) == ALIGN
    for part in ("q", "k"):
        def f(dtype=0, **kw):
            return rotary(L, dtype, **{part: hd(**kw)})
        assert f(x=None) == NULL and f(y=None) == NULL
        assert f(x=A + 1) == ALIGN and f(y=A + 1) == ALIGN and f(dtype=1, x=A + 2) == ALIGN
        assert f(heads=-1) == SHAPE and f(heads=(1 << 20) + 1) == SHAPE
        assert f(ldx=-1) == SHAPE and f(hsx=-64) == SHAPE
        assert f(ldx=1 << 58) == SHAPE
        # outputs that share elements: heads, tokens, or both axes with one stride
        assert f(hsy=63) == SHAPE and f(ldy=255) == SHAPE and f(ldy=64) == SHAPE
        assert f(ldy=0) == SHAPE and f(hsy=0) == SHAPE
        # in place with other strides
        assert f(y=A, ldy=512) == UNSUP and f(y=A, ldx=64, hsx=256, ldy=256, hsy=64) == UNSUP
    # nothing to do needs no buffers
    assert rotary(L, T=0, q=hd(None, None), pos=None, freqs=None) == OK
    assert rotary(L, q=hd(None, None, 0), pos=None, freqs=None) == OK
    assert rotary(L, q=hd(y=A), rot=0, pos=None, freqs=None) == OK


def test_rotary_frequencies(L):
    f, m = aqfq.aqfq_rotary_freqs(8, base=100.0)
    want = torch.tensor([100.0 ** (-i / 4) for i in range(4)], dtype=torch.float64)
    assert m == 1.0 and float((f / want - 1).abs().max()) < 1e-14
    g, m = aqfq.aqfq_rotary_freqs(8, base=100.0, scaling=aqfq.ROTARY_LINEAR, factor=4.0)
    assert m == 1.0 and float((g * 4 / want - 1).abs().max()) < 1e-14
    # the last pair is interpolated in full, the first one kept
    g, m = aqfq.aqfq_rotary_freqs(8, base=100.0, scaling=aqfq.ROTARY_NTK, factor=4.0)
    assert m == 1.0 and abs(float(g[0]) - 1) < 1e-14 and abs(float(g[3] * 4 / want[3]) - 1) < 1e-13
    # turns over the length: 1000 / 2 pi = 159, 50, 15.9, 5.03; kept above 40, divided below 10
    g, m = aqfq.aqfq_rotary_freqs(8, base=100.0, scaling=aqfq.ROTARY_PARTS, factor=4.0, length=1000.0,
                                  low=10.0, high=40.0)
    k = (1000 * float(want[2]) / (2 * math.pi) - 10) / 30
    assert 0 < k < 1
    parts = torch.tensor([1, 1, k + (1 - k) / 4, 0.25], dtype=torch.float64) * want
    assert float((g / parts - 1).abs().max()) < 1e-13 and abs(m - (0.1 * math.log(4) + 1)) < 1e-7
    f, m = aqfq.aqfq_rotary_freqs(0)
    assert len(f) == 0
    buf = (ctypes.c_double * 64)()
    p = ctypes.addressof(buf)
    g = lambda rot=8, base=1e4, s=0, factor=4.0, length=1e3, low=1.0, high=32.0, out=p: L.aqfq_rotary_freqs(
        rot, base, s, factor, length, low, high, out, None)
    assert g() == OK and g(rot=7) == SHAPE and g(rot=-2) == SHAPE and g(out=None) == NULL
    assert g(rot=8194) == SHAPE
    assert g(base=0.0) == SHAPE and g(base=float("nan")) == SHAPE and g(base=float("inf")) == SHAPE
    assert g(s=4) == UNSUP and g(s=-1) == UNSUP
    for s in (1, 2, 3):
        assert g(s=s, factor=0.5) == SHAPE and g(s=s, factor=float("nan")) == SHAPE and g(s=s) == OK
    assert g(s=3, length=0.0) == SHAPE and g(s=3, low=32.0) == SHAPE and g(s=3, high=float("nan")) == SHAPE


def test_rotary_binding_checks():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos, freqs = torch.zeros(4, dtype=torch.int64), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        aqfq.aqfq_rotary(q, pos, freqs, torch.empty_like(q))
    with pytest.raises(ValueError, match="heads"):
        aqfq.aqfq_rotary(q[0], pos, freqs, q)


# ---- norms, gate and residual between two blocks ---------------------------------------

def jfwd(L, dtype=0, x=A, ldx=64, f=2 * A, ldf=64, R=4, C=64, post=1, pd=0, gp=A, gate=A, gn=A, eps=1e-6,
         h=3 * A, ldh=64, y=4 * A, ldy=64, rp=A, rq=A):
    return L.aqfq_block_norm_fwd(dtype, x, ldx, f, ldf, R, C, post, pd, gp, gate, 1.0, gn, eps, h, ldh, y, ldy,
                                 rp, rq, None)


def test_block_norm_fwd_checks(L):
    assert jfwd(L, dtype=2) == UNSUP and jfwd(L, pd=-1) == UNSUP
    assert jfwd(L, C=0) == SHAPE and jfwd(L, C=-1) == SHAPE and jfwd(L, R=-1) == SHAPE
    for ld in ("ldx", "ldf", "ldh", "ldy"):
        assert jfwd(L, **{ld: 63}) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert jfwd(L, eps=eps) == SHAPE
    assert jfwd(L, x=None, f=None, post=0, gp=None, gate=None, rp=None) == NULL
    assert jfwd(L, h=None, y=None) == NULL
    assert jfwd(L, y=None) == NULL and jfwd(L, y=None, gn=None) == NULL     # a norm that is not taken
    assert jfwd(L, post=0) == UNSUP and jfwd(L, post=0, gp=None) == UNSUP and jfwd(L, post=0, rp=None) == UNSUP
    assert jfwd(L, f=None) == NULL and jfwd(L, f=None, post=0, gp=None, rp=None) == NULL
    for p in ("x", "f", "h", "y"):
        assert jfwd(L, **{p: A + 1}) == ALIGN and jfwd(L, dtype=1, **{p: A + 2}) == ALIGN
    for p in ("gp", "gate", "gn"):
        assert jfwd(L, **{p: A + 1}) == ALIGN and jfwd(L, pd=1, **{p: A + 2}) == ALIGN
    assert jfwd(L, rp=A + 2) == ALIGN and jfwd(L, rq=A + 2) == ALIGN
    assert jfwd(L, R=0, x=None, f=None, h=None, y=None) == OK


def jbwd(L, dtype=0, dy=A, lddy=64, dh=A, lddh=64, h=A, ldh=64, f=A, ldf=64, R=64, C=64, rp=A, rq=A, pd=0, gp=A,
         gate=A, gn=A, dx=2 * A, lddx=64, df=3 * A, lddf=64, dgp=None, dga=None, dgn=None, ws=None, wsb=0):
    return L.aqfq_block_norm_bwd(dtype, dy, lddy, dh, lddh, h, ldh, f, ldf, R, C, rp, rq, pd, gp, gate, 1.0, gn,
                                 dx, lddx, df, lddf, dgp, dga, dgn, 0, ws, wsb, None)


def test_block_norm_bwd_checks(L):
    assert jbwd(L, dtype=3) == UNSUP and jbwd(L, pd=2) == UNSUP
    assert jbwd(L, C=0) == SHAPE and jbwd(L, R=-1) == SHAPE
    for ld in ("lddy", "lddh", "ldh", "ldf", "lddx", "lddf"):
        assert jbwd(L, **{ld: 63}) == SHAPE
    assert jbwd(L, dx=None, df=None) == NULL
    assert jbwd(L, dy=None, dh=None) == NULL
    assert jbwd(L, h=None) == NULL and jbwd(L, rq=None) == NULL
    assert jbwd(L, dy=None) == NULL and jbwd(L, dy=None, gn=None, dgn=A, ws=A, wsb=1 << 20) == NULL
    assert jbwd(L, f=None) == NULL and jbwd(L, f=None, df=None, rp=None, gp=None) == NULL
    assert jbwd(L, f=None, df=None, rp=None, gp=None, gate=None, dga=A, ws=A, wsb=1 << 20) == NULL
    assert jbwd(L, rp=None) == UNSUP and jbwd(L, rp=None, gp=None, dgp=A, ws=A, wsb=1 << 20) == UNSUP
    for p in ("dy", "dh", "h", "f", "dx", "df"):
        assert jbwd(L, **{p: A + 1}) == ALIGN
    for p in ("gp", "gate", "gn"):
        assert jbwd(L, **{p: A + 1}) == ALIGN
    need = aqfq.aqfq_block_norm_bwd_workspace_bytes(64, 64)
    assert need > 0
    for p in ("dgp", "dga", "dgn"):
        assert jbwd(L, **{p: A + 2}, ws=A, wsb=need) == ALIGN
        assert jbwd(L, **{p: A}) == WS and jbwd(L, **{p: A}, ws=A, wsb=need - 1) == WS
        assert jbwd(L, **{p: A}, ws=A + 4, wsb=need) == ALIGN
    assert jbwd(L, R=0, dy=None, dh=None, h=None, f=None, rp=None, rq=None, dx=None, df=None) == OK
    assert (aqfq.aqfq_block_norm_bwd_workspace_bytes(10 ** 7, 64)
            == aqfq.aqfq_block_norm_bwd_workspace_bytes(10 ** 8, 64))
    assert aqfq.aqfq_block_norm_bwd_workspace_bytes(-1, 64) == 0


def test_block_norm_binding_checks():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        aqfq.aqfq_block_norm_fwd(t, t, 1e-6, h=t)
    with pytest.raises(ValueError, match="missing"):
        aqfq.aqfq_block_norm_fwd(None, None, 1e-6, h=t)
    with pytest.raises(ValueError, match="missing"):
        aqfq.aqfq_block_norm_bwd(None, None, t, t, dx=t)


# ---- gated product ---------------------------------------------------------------------

def ck(fmt=aqfq.INT8, group=128, codes=7 * A, scale=8 * A):
    return ctypes.byref(aqfq.Ckpt8(fmt, group, codes, scale))


def gfwd(L, x=A, ldx=64, w=2 * A, ldw=64, M=4, N=32, K=64, act=4, y=3 * A, ldy=32, gate=None, up=None, ws=None,
         wsb=0, err=None):
    return L.aqfq_gated_fwd(x, ldx, w, ldw, M, N, K, act, y, ldy, gate, up, ws, wsb, err, None)


def gdgrad(L, x=A, ldx=32, w=2 * A, ldw=64, M=4, N=32, K=64, act=4, gate="ok", up="ok", y=3 * A, ldy=128, h=None,
           ldh=0, ws=None, wsb=0, err=None):
    return L.aqfq_gated_dgrad(x, ldx, w, ldw, M, N, K, act, ck() if gate == "ok" else gate,
                              ck() if up == "ok" else up, y, ldy, h, ldh, ws, wsb, err, None)


def test_gated_checks(L):
    for f in (gfwd, gdgrad):
        assert f(L, x=None) == NULL and f(L, w=None) == NULL and f(L, y=None) == NULL
        assert f(L, x=A + 8) == ALIGN and f(L, w=A + 2) == ALIGN and f(L, y=A + 1) == ALIGN
        assert f(L, ldx=68) == ALIGN and f(L, ldw=68) == ALIGN
        assert f(L, ldx=24) == SHAPE and f(L, ldw=56) == SHAPE and f(L, ldy=24) == SHAPE
        assert f(L, M=-1) == SHAPE and f(L, N=1 << 30) == SHAPE and f(L, K=-8) == SHAPE
        assert f(L, act=5) == UNSUP and f(L, act=-1) == UNSUP
        assert f(L, err=A + 2) == ALIGN
        assert f(L, gate=ck(), up=None) == NULL and f(L, gate=None, up=ck()) == NULL
        assert f(L, gate=ck(group=16), up=ck(group=16)) == UNSUP
        assert f(L, gate=ck(), up=ck(group=64)) == UNSUP
        assert f(L, gate=ck(), up=ck(fmt=aqfq.FP8_E4M3)) == UNSUP
        assert f(L, gate=ck(codes=None), up=ck()) == NULL
    assert gfwd(L, N=1 << 29, ldy=1 << 29) == SHAPE               # 2N beyond the limit
    assert gdgrad(L, ldy=64) == SHAPE                             # dp has 2K columns
    assert gdgrad(L, gate=None, up=None) == NULL                  # the gradient needs what was kept
    assert gdgrad(L, h=A, ldh=32) == SHAPE and gdgrad(L, h=A + 1, ldh=64) == ALIGN
    need = aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_FWD, 70, 300, 33000)
    big = dict(M=70, N=300, K=33000, ldx=33000, ldw=33000, ldy=300)
    assert need > 0 and gfwd(L, **big) == WS and gfwd(L, ws=A, wsb=need - 1, **big) == WS
    assert gfwd(L, ws=A + 8, wsb=need, **big) == ALIGN
    assert gfwd(L, M=0, x=None, w=None, y=None) == OK and gfwd(L, N=0, x=None, w=None, y=None) == OK
    none = ck(codes=None, scale=None)
    assert gdgrad(L, M=0, x=None, w=None, y=None, gate=none, up=none) == OK
    assert aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_WGRAD, 70, 300, 33000) == 0
    assert aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_FWD, -1, 300, 33000) == 0


def gbwd(L, gate="ok", up="ok", act=4, dtype=0, dy=A, lddy=64, R=4, C=64, dp=2 * A, lddp=128, y=3 * A, ldy=64):
    return L.aqfq_ckpt8_gated_bwd(ck() if gate == "ok" else gate, ck() if up == "ok" else up, act, dtype, dy, lddy, R,
                                  C, dp, lddp, y, ldy, None)


def test_elementwise_gated_gradient_checks(L):
    assert gbwd(L, gate=None) == NULL and gbwd(L, up=None) == NULL
    assert gbwd(L, up=ck(group=32)) == UNSUP and gbwd(L, up=ck(fmt=aqfq.FP8_E4M3)) == UNSUP
    assert gbwd(L, act=5) == UNSUP and gbwd(L, dtype=2) == UNSUP
    assert gbwd(L, dp=None, y=None) == NULL and gbwd(L, dy=None) == NULL
    for p in ("dy", "dp", "y"):
        assert gbwd(L, **{p: A + 1}) == ALIGN
    assert gbwd(L, lddy=63) == SHAPE and gbwd(L, lddp=127) == SHAPE and gbwd(L, ldy=63) == SHAPE
    assert gbwd(L, R=-1) == SHAPE and gbwd(L, C=-1) == SHAPE
    none = ck(codes=None, scale=None)
    assert gbwd(L, gate=none, up=none, R=0, dy=None, dp=None, y=None) == OK


def test_gated_binding_checks():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        aqfq.aqfq_gated_fwd(t, t, t)

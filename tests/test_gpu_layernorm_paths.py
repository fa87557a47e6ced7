"""Layer norm where the kernel is chosen by the size: every class of widths, aligned and not, for
one row, a cluster's and many; workspaces at every alignment that the
header allows; rows whose mean times 1 / deviation overflows; the rings that serve many rows, at
the least rows that take them and with every stage reused.  Bounds as in test_gpu_layernorm.py."""
import pytest
import torch

from layerlib import DEV, FMTS, Framed, grid_values, kept, new_ckpt, pack_ref, randn, ws
from learnable_scale_fake_gb300 import aqfq
from test_gpu_layernorm import EPS, _case, _check_bwd, _check_fwd, _stats

pytestmark = pytest.mark.gpu


# rows in registers with one group of warps per block (sums straight to scratch), several
# groups, odd widths, and both kinds of the ring
@pytest.mark.parametrize("R,C", [(60, 1160), (200, 4096), (20, 8192), (400, 512), (90, 1003),
                                 (700, 8192), (1300, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["none", "int8"])
def test_backward_workspace_at_any_multiple_of_8_bytes(R, C, dtype, fmt):
    x, g, _ = _case(R, C, R + C, dtype)
    dy = randn((R, C), R, dtype=dtype)
    mu, rs = _stats(x)
    m, r = mu[:, 0].float().to(DEV), rs[:, 0].float().to(DEV)
    xd, ck, kx = x.to(DEV), None, x
    if fmt != "none":
        ck, codes, scale = new_ckpt(R, C, fmt, 64)
        aqfq.aqfq_ckpt8_pack(ck, xd)
        torch.cuda.synchronize()
        kx, xd = kept(codes, scale, fmt, 64), None
    need = aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C)
    buf = torch.empty(need + 64, dtype=torch.uint8, device=DEV)
    first = None
    for off in (0, 8, 16, 24):
        buf.fill_(0xA5)
        dx, dg, db = torch.empty(R, C, dtype=dtype, device=DEV), *torch.empty(2, C, device=DEV)
        aqfq.aqfq_layernorm_bwd(dy.to(DEV), xd, m, r, g.to(DEV), dx, dgamma=dg, dbeta=db, ckpt=ck,
                                workspace=buf[off:off + need])
        torch.cuda.synchronize()
        assert bool((buf[:off] == 0xA5).all()) and bool((buf[off + need:] == 0xA5).all())
        if first is None:
            first = (dx, dg, db)
            _check_bwd(kx, dy, m, r, g, None, dx, dg, db)
        assert all(torch.equal(a, b) for a, b in zip(first, (dx, dg, db)))


# widths that fill their lanes and ones that leave some beyond the row, aligned and odd
@pytest.mark.parametrize("C", [8, 32, 64, 256, 512, 1024, 2048])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows_of_a_large_value(C, pad, dtype):
    """x - mean is zero all over the row: dx = rstd (dy gamma - mean(dy gamma)) and dgamma = 0
    though mean rstd is beyond binary32 (the widths are powers of two, so the mean is exact)."""
    R, big = 5, 1.5 * 2.0 ** 121
    rows = lambda t: torch.cat([t, torch.zeros(R, pad, dtype=t.dtype)], 1).to(DEV)[:, :C]
    x, dy = torch.full((R, C), big, dtype=dtype), randn((R, C), C, dtype=dtype)
    _, g, _ = _case(R, C, 5, dtype)
    m, r = torch.full((R,), big, device=DEV), torch.full((R,), 316.0, device=DEV)
    dx, dg, db = torch.empty(R, C, dtype=dtype, device=DEV), *torch.empty(2, C, device=DEV)
    w = torch.empty(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
    aqfq.aqfq_layernorm_bwd(rows(dy), rows(x), m, r, g.to(DEV), dx, dgamma=dg, dbeta=db, workspace=w)
    torch.cuda.synchronize()
    _check_bwd(x, dy, m, r, g, None, dx, dg, db)
    assert bool((dg == 0).all())


BF16, F32 = torch.bfloat16, torch.float32


def ckpt_at(rows, cols, fmt, group, off):
    """A checkpoint whose codes start `off` bytes into a buffer that is aligned to 256."""
    buf = torch.full((rows * cols + off,), 0x5A, dtype=torch.uint8, device=DEV)
    codes = buf[off:].view(rows, cols)
    scale = torch.full((rows, -(-cols // group)), -7.0, device=DEV)
    return aqfq.ckpt8(FMTS[fmt], group, codes, scale), codes, scale


# Two rows per stage; 4, 8 or 16 warps per row.  The second of each pair of sizes has more turns
# than stages and, with 16 columns per lane, a lane with only its first 8 in the row.
@pytest.mark.parametrize("R,C,warps", [(4865, 1104, 4), (15809, 1032, 4), (2433, 4096, 8), (4257, 4088, 8),
                                       (1217, 8192, 16), (2129, 8184, 16), (2130, 4112, 16)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", [None, ("int8", 128), ("e4m3", 32), ("int8", 64)])
def test_forward_ring(R, C, warps, dtype, form):
    assert aqfq.aqfq_selftest_layernorm_ring(False, dtype, R, C) == warps
    x, g, b = _case(R, C, R, dtype)
    i = 0 if form is None else form[1] // 32
    pad = (0, 8, 16)[i % 3]
    fx, fy = Framed(R, C, dtype, pad, pad, x), Framed(R, C, dtype, pad, pad)
    m, r = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    ck, codes, scale = ckpt_at(R, C, *form, 8 if i == 2 else 0) if form else (None, None, None)
    pd = F32 if i % 2 else BF16
    g, b = g.to(pd), b.to(pd)
    aqfq.aqfq_layernorm_fwd(fx.view, g.to(DEV), b.to(DEV), EPS, fy.view, mean=m, rstd=r, ckpt=ck)
    torch.cuda.synchronize()
    _check_fwd(x, g, b, fy.view, m, r)
    assert fy.intact()
    if form:
        q, s = pack_ref(x, *form)
        assert (scale.cpu().numpy() == s).all() and (grid_values(codes, form[0]) == q).all()
        # without parameters and statistics: the same rows and codes
        y, (ck2, codes2, scale2) = torch.empty(R, C, dtype=dtype, device=DEV), ckpt_at(R, C, *form, 0)
        aqfq.aqfq_layernorm_fwd(fx.view, torch.ones(C, dtype=pd, device=DEV), None, EPS, y, ckpt=ck2)
        y2 = torch.empty(R, C, dtype=dtype, device=DEV)
        aqfq.aqfq_layernorm_fwd(fx.view, None, None, EPS, y2)
        torch.cuda.synchronize()
        assert torch.equal(codes, codes2) and torch.equal(scale, scale2) and torch.equal(y, y2)


def test_forward_ring_non_finite_rows_stay_alone():
    R, C = 1217, 8192
    assert aqfq.aqfq_selftest_layernorm_ring(False, BF16, R, C) == 16
    x, g, b = _case(R, C, 77, BF16)
    x[5, 3], x[1216, 8191], x[700, 4096] = float("nan"), float("inf"), -float("inf")
    y, m, r = torch.empty(R, C, dtype=BF16, device=DEV), torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    aqfq.aqfq_layernorm_fwd(x.to(DEV), g.to(DEV), b.to(DEV), EPS, y, mean=m, rstd=r)
    torch.cuda.synchronize()
    bad = torch.zeros(R, dtype=torch.bool)
    bad[[5, 700, 1216]] = True
    assert torch.equal(torch.isnan(y.cpu()).any(1), bad) and bool(torch.isnan(y.cpu()[bad]).all())
    _check_fwd(x[~bad], g, b, y.cpu()[~bad], m.cpu()[~bad], r.cpu()[~bad])


def _bwd(R, C, dtype, form, with_dres, accumulate, pad, warps):
    got = aqfq.aqfq_selftest_layernorm_ring(True, dtype, R, C, form is not None, with_dres)
    assert got == warps
    x, g, _ = _case(R, C, R + 1, dtype)
    dy = randn((R, C), R + 2, dtype=dtype)
    dres = randn((R, C), R + 3, dtype=dtype) if with_dres else None
    mu, rs = _stats(x)
    m, r = mu[:, 0].float().to(DEV), rs[:, 0].float().to(DEV)
    fd, fo = Framed(R, C, dtype, pad, pad, dy), Framed(R, C, dtype, pad, 0)
    fr = Framed(R, C, dtype, 0, pad, dres) if with_dres else None
    fx, ck, kx = Framed(R, C, dtype, pad, pad, x), None, x
    if form:
        ck, codes, scale = new_ckpt(R, C, *form)
        aqfq.aqfq_ckpt8_pack(ck, fx.view)
        torch.cuda.synchronize()
        kx = kept(codes, scale, *form)
    base = 0.5 if accumulate else 0.0
    dg, db = torch.full((2, C), 0.5 if accumulate else float("nan"), device=DEV)
    w = ws(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C))
    args = (fd.view, None if form else fx.view, m, r, g.to(DEV))
    kw = dict(dres=None if fr is None else fr.view, ckpt=ck, workspace=w)
    aqfq.aqfq_layernorm_bwd(*args, fo.view, dgamma=dg, dbeta=db, accumulate=accumulate, **kw)
    # the input gradient alone, the column sums alone
    dx2 = torch.empty(R, C, dtype=dtype, device=DEV)
    aqfq.aqfq_layernorm_bwd(*args, dx2, **kw)
    torch.cuda.synchronize()
    _check_bwd(kx, dy, m, r, g, dres, fo.view, dg, db, base)
    assert fo.intact() and torch.equal(dx2, fo.view)
    if not with_dres:
        dg2, db2 = torch.full((2, C), base, device=DEV)
        aqfq.aqfq_layernorm_bwd(*args, None, dgamma=dg2, dbeta=db2, accumulate=accumulate, **kw)
        torch.cuda.synchronize()
        assert torch.equal(dg, dg2) and torch.equal(db, db2)


# one to 16 warps per row; the second of each pair of sizes has more turns than stages, and
# widths of an odd number of 8 columns where x is kept as it is
BWD = [(9729, 512, 1), (14593, 496, 1), (4865, 1008, 2), (8513, 1024, 2), (2433, 2048, 4), (4257, 1040, 4),
       (1217, 4096, 8), (2129, 2064, 8), (609, 8192, 16), (1065, 4112, 16)]


@pytest.mark.parametrize("R,C,warps", BWD)
@pytest.mark.parametrize("form", [None, ("int8", 128), ("e4m3", 32)])
@pytest.mark.parametrize("with_dres", [False, True])
def test_backward_ring_bf16(R, C, warps, form, with_dres):
    cols = C - 8 if form is None and (C - 8) * 2 > 32 * 16 * warps else C
    _bwd(R, cols, BF16, form, with_dres, accumulate=with_dres == (form is None), pad=8 if with_dres else 0,
         warps=warps)


@pytest.mark.parametrize("R,C,warps", BWD)
@pytest.mark.parametrize("form", [None, ("int8", 64), ("e4m3", 32)])
def test_backward_ring_fp32(R, C, warps, form):
    _bwd(R, C, F32, form, False, accumulate=form is None, pad=8, warps=warps)


def test_rings_give_the_same_bits_again_and_on_another_stream():
    R, C = 2433, 4096
    x, g, b = _case(R, C, 81, BF16)
    xd, gd, bd, dy = x.to(DEV), g.to(DEV), b.to(DEV), randn((R, C), 82).to(DEV)
    out = []
    for st in (None, torch.cuda.Stream(), None):
        y, dx = torch.empty_like(xd), torch.empty_like(xd)
        m, r, dg, db = (torch.empty(n, device=DEV) for n in (R, R, C, C))
        w = ws(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C))
        torch.cuda.synchronize()
        aqfq.aqfq_layernorm_fwd(xd, gd, bd, EPS, y, mean=m, rstd=r, stream=st)
        aqfq.aqfq_layernorm_bwd(dy, xd, m, r, gd, dx, dgamma=dg, dbeta=db, workspace=w, stream=st)
        torch.cuda.synchronize()
        out.append((y, m, r, dx, dg, db))
    for o in out[1:]:
        assert all(torch.equal(p, q) for p, q in zip(out[0], o))


# both ends of the classes of columns that have kernels of their own, up to the widths that a
# block walks; pad 1: rows that allow no wide access
@pytest.mark.parametrize("C", [120, 128, 256, 264, 384, 512, 520, 1024, 1032, 1536, 2048, 3000, 4096, 4104, 6000,
                               8192, 8200, 12288, 16384, 16392])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_class_of_widths(C, pad, dtype):
    for k, R in enumerate((1, 7, 61, 400)):
        x, g, b = _case(R, C, 3 * C + R, dtype)
        fmt, group = (("int8", 32), ("e4m3", 128))[k % 2]
        fx, fy = Framed(R, C, dtype, pad, pad, x), Framed(R, C, dtype, pad, pad)
        m, r = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
        ck, codes, scale = new_ckpt(R, C, fmt, group)
        aqfq.aqfq_layernorm_fwd(fx.view, g.to(DEV), b.to(DEV), EPS, fy.view, mean=m, rstd=r, ckpt=ck)
        torch.cuda.synchronize()
        _check_fwd(x, g, b, fy.view, m, r)
        q, s = pack_ref(x, fmt, group)
        assert fy.intact() and (scale.cpu().numpy() == s).all() and (grid_values(codes, fmt) == q).all()
        dy, dres = randn((R, C), C + R, dtype=dtype), randn((R, C), C + R + 1, dtype=dtype)
        fd, fo = Framed(R, C, dtype, pad, pad, dy), Framed(R, C, dtype, pad, pad)
        w = ws(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C))
        for from_ck in (False, True):
            dg, db = torch.full((2, C), float("nan"), device=DEV)
            aqfq.aqfq_layernorm_bwd(fd.view, None if from_ck else fx.view, m, r, g.to(DEV), fo.view, dgamma=dg,
                                    dbeta=db, dres=dres.to(DEV) if k % 2 else None,
                                    ckpt=ck if from_ck else None, workspace=w)
            torch.cuda.synchronize()
            kx = kept(codes, scale, fmt, group) if from_ck else x
            _check_bwd(kx, dy, m, r, g, dres if k % 2 else None, fo.view, dg, db)
            assert fo.intact()

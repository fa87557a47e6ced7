"""Layer norm forward and backward against 64-bit formulas.

Bounds (U the unit roundoff of binary32): a sum over C columns is at most
D = C / 256 + 64 roundings deep, so the mean is D U mean|x| off and the variance
relatively (D + 8) U plus the square of the mean's error over the deviation;
y and dx follow from their factors; a column sum over R rows is at most
R + 64 roundings deep; a stored BF16 value is rounded once more."""
import pytest
import torch

from layerlib import BF, DEV, Framed, U, close, grid_values, kept, new_ckpt, pack_ref, randn, ws
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 8), (64, 100), (2, 255), (300, 256), (33, 1003), (7, 2056),
          (1000, 768), (5, 5000), (3, 8192), (2, 20000), (2, 70001)]
EPS = 1e-5


def _case(R, C, seed, dtype):
    x = randn((R, C), seed, dtype=torch.float32)
    x[:, ::61] *= 20.0
    x += 0.5
    return (x.to(dtype), (1 + randn((C,), seed + 1, 0.2, torch.float32)),
            randn((C,), seed + 2, 0.5, torch.float32))


def _stats(x, eps=EPS):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    return mu, 1.0 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + eps)


def _check_fwd(x, g, b, y, mean, rstd, eps=EPS):
    R, C = x.shape
    D = C / 256 + 64
    xd = x.double()
    mu, rs = _stats(x, eps)
    g = torch.ones(C).double() if g is None else g.double()
    b = torch.zeros(C).double() if b is None else b.double()
    emu = D * U * xd.abs().mean(1, keepdim=True)
    ers = (D + 8) * U + (emu * rs) ** 2  # relative
    close(mean, mu[:, 0], emu[:, 0], "mean")
    close(rstd, rs[:, 0], (ers * rs)[:, 0], "rstd")
    t = (xd - mu) * rs * g
    ref = t + b
    tol = emu * rs * g.abs() + t.abs() * (ers + 4 * U) + U * (b.abs() + ref.abs())
    if x.dtype == torch.bfloat16:
        tol = tol + BF * ref.abs()
    close(y, ref, tol, f"y {R}x{C}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pdtype", [torch.bfloat16, torch.float32])
def test_forward(dtype, pdtype):
    for i, (R, C) in enumerate(SHAPES):
        x, g, b = _case(R, C, 10 * i, dtype)
        g, b = g.to(pdtype), b.to(pdtype)
        for pad, off in ((0, 0), (8, 8), (3, 1)):
            fx, fy = Framed(R, C, dtype, pad, off, x), Framed(R, C, dtype, pad, off)
            m, r = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
            aqfq.aqfq_layernorm_fwd(fx.view, g.to(DEV), b.to(DEV), EPS, fy.view, mean=m, rstd=r)
            torch.cuda.synchronize()
            _check_fwd(x, g, b, fy.view, m, r)
            assert fy.intact()


def test_forward_without_parameters_and_statistics():
    x, _, _ = _case(9, 640, 3, torch.float32)
    m, r, y, y2 = (torch.empty(9, device=DEV), torch.empty(9, device=DEV),
                   torch.empty(9, 640, device=DEV), torch.empty(9, 640, device=DEV))
    aqfq.aqfq_layernorm_fwd(x.to(DEV), None, None, EPS, y, mean=m, rstd=r)
    aqfq.aqfq_layernorm_fwd(x.to(DEV), None, None, EPS, y2)
    torch.cuda.synchronize()
    _check_fwd(x, None, None, y, m, r)
    assert torch.equal(y, y2)


def test_forward_large_mean_and_constant_rows():
    """A mean a thousand deviations away, rows of one value, eps zero."""
    x = randn((6, 4096), 4, dtype=torch.float32) + 1000.0
    x[2] = 3.25
    m, r, y = torch.empty(6, device=DEV), torch.empty(6, device=DEV), torch.empty(6, 4096, device=DEV)
    aqfq.aqfq_layernorm_fwd(x.to(DEV), None, None, EPS, y, mean=m, rstd=r)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 3, 4, 5])
    _check_fwd(x[rows], None, None, y.cpu()[rows], m.cpu()[rows], r.cpu()[rows])
    assert bool((y[2] == 0).all()) and float(m[2]) == 3.25
    x = x[rows].contiguous()
    y, m, r = y[:5].contiguous(), m[:5].contiguous(), r[:5].contiguous()
    aqfq.aqfq_layernorm_fwd(x.to(DEV), None, None, 0.0, y, mean=m, rstd=r)
    torch.cuda.synchronize()
    _check_fwd(x, None, None, y, m, r, 0.0)


def test_non_finite_rows_stay_alone():
    x, g, b = _case(5, 1000, 5, torch.float32)
    x[1, 3], x[3, 999] = float("nan"), float("inf")
    y, m, r = torch.empty(5, 1000, device=DEV), torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    ck, codes, scale = new_ckpt(5, 1000, "int8", 128)
    aqfq.aqfq_layernorm_fwd(x.to(DEV), g.to(DEV), b.to(DEV), EPS, y, mean=m, rstd=r, ckpt=ck)
    dy = randn((5, 1000), 6, dtype=torch.float32)
    dx = torch.empty(5, 1000, device=DEV)
    aqfq.aqfq_layernorm_bwd(dy.to(DEV), None, m, r, g.to(DEV), dx, ckpt=ck)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 2, 4])
    assert bool(torch.isnan(y[[1, 3]]).all()) and bool(torch.isnan(dx[[1, 3]]).all())
    assert bool(torch.isfinite(dx.cpu()[rows]).all())
    _check_fwd(x[rows], g, b, y.cpu()[rows], m.cpu()[rows], r.cpu()[rows])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,group", [("int8", 128), ("e4m3", 32), ("int8", 64)])
def test_forward_checkpoint_is_the_packed_input(dtype, fmt, group):
    for i, (R, C) in enumerate(SHAPES):
        x, g, b = _case(R, C, 500 + i, dtype)
        fx, fy = Framed(R, C, dtype, i % 2, i % 3, x), Framed(R, C, dtype)
        ck, codes, scale = new_ckpt(R, C, fmt, group)
        m, r = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
        aqfq.aqfq_layernorm_fwd(fx.view, g.to(DEV), b.to(DEV), EPS, fy.view, mean=m, rstd=r, ckpt=ck)
        torch.cuda.synchronize()
        q, s = pack_ref(x, fmt, group)
        assert (scale.cpu().numpy() == s).all() and (grid_values(codes, fmt) == q).all()
        _check_fwd(x, g, b, fy.view, m, r)


def _check_bwd(kept_x, dy, m, r, g, dres, dx, dg, db, base=0.0):
    R, C = dy.shape
    D = C / 256 + 64
    m, r = m.double().cpu()[:, None], r.double().cpu()[:, None]
    g = torch.ones(C).double() if g is None else g.double()
    h, d = (kept_x.double() - m) * r, dy.double()
    # h as the kernel forms it: two roundings, the first of the size of x - mean
    eh = 2 * U * h.abs() + U * (kept_x.double() - m).abs() * r
    u = d * g
    m1, m2 = u.mean(1, keepdim=True), (u * h).mean(1, keepdim=True)
    if dx is not None:
        ref = r * (u - m1 - h * m2)
        e1 = D * U * u.abs().mean(1, keepdim=True)
        e2 = (D * U * (u * h).abs() + u.abs() * eh).mean(1, keepdim=True)
        size = u.abs() + m1.abs() + (h * m2).abs()
        tol = r * (e1 + h.abs() * e2 + eh * m2.abs() + 4 * U * size)
        if dres is not None:
            ref = ref + dres.double()
        tol = tol + U * ref.abs() + (BF * ref.abs() if dy.dtype == torch.bfloat16 else 0)
        close(dx, ref, tol, f"dx {R}x{C}")
    deep = (R + 64) * U
    if dg is not None:
        close(dg, (d * h).sum(0) + base,
              (deep * (d * h).abs() + d.abs() * eh).sum(0) + deep * abs(base), "dgamma")
    if db is not None:
        close(db, d.sum(0) + base, deep * (d.abs().sum(0) + abs(base)), "dbeta")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,group", [("none", 0), ("int8", 128), ("e4m3", 64), ("int8", 32)])
def test_backward(dtype, pdtype, fmt, group):
    for i, (R, C) in enumerate(SHAPES):
        x, g, _ = _case(R, C, 900 + i, dtype)
        g = g.to(pdtype)
        dy, dres = randn((R, C), 1000 + i, dtype=dtype), randn((R, C), 1100 + i, dtype=dtype)
        mu, rs = _stats(x)
        m, r = mu[:, 0].float().to(DEV), rs[:, 0].float().to(DEV)
        odd, acc = i % 3 == 1, i % 2 == 1
        fd = Framed(R, C, dtype, 3 if odd else 0, 1 if odd else 0, dy)
        fr, fo = Framed(R, C, dtype, 0, 0, dres), Framed(R, C, dtype, 8, 8)
        fg, fb = Framed(1, C, torch.float32), Framed(1, C, torch.float32)
        fg.view.fill_(0.5 if acc else float("nan"))
        fb.view.fill_(0.5 if acc else float("nan"))
        w = ws(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C))
        xd, ck, kx = x.to(DEV), None, x
        if fmt != "none":
            ck, codes, scale = new_ckpt(R, C, fmt, group)
            aqfq.aqfq_ckpt8_pack(ck, xd)
            torch.cuda.synchronize()
            kx, xd = kept(codes, scale, fmt, group), None
        aqfq.aqfq_layernorm_bwd(fd.view, xd, m, r, g.to(DEV), fo.view, dgamma=fg.view[0],
                                dbeta=fb.view[0], dres=fr.view if i % 2 else None, ckpt=ck,
                                accumulate=acc, workspace=w)
        torch.cuda.synchronize()
        _check_bwd(kx, dy, m, r, g, dres if i % 2 else None, fo.view, fg.view[0], fb.view[0],
                   0.5 if acc else 0.0)
        assert fo.intact() and fg.intact() and fb.intact()


def test_backward_parts_alone():
    x, g, _ = _case(200, 1160, 31, torch.bfloat16)
    dy = randn((200, 1160), 32).to(DEV)
    mu, rs = _stats(x)
    m, r, xd, gd = mu[:, 0].float().to(DEV), rs[:, 0].float().to(DEV), x.to(DEV), g.to(DEV)
    w = ws(aqfq.aqfq_layernorm_bwd_workspace_bytes(200, 1160))
    new = lambda: torch.empty(1160, device=DEV)
    dx, dx2, a, b, a2, b2 = torch.empty_like(dy), torch.empty_like(dy), new(), new(), new(), new()
    aqfq.aqfq_layernorm_bwd(dy, xd, m, r, gd, dx, dgamma=a, dbeta=b, workspace=w)
    aqfq.aqfq_layernorm_bwd(dy, xd, m, r, gd, dx2)
    aqfq.aqfq_layernorm_bwd(dy, xd, m, r, gd, None, dgamma=a2, workspace=w)
    aqfq.aqfq_layernorm_bwd(dy, xd, m, r, gd, None, dbeta=b2, workspace=w)
    torch.cuda.synchronize()
    for got in ((dx, a, b), (dx2, a2, b2)):
        _check_bwd(x, dy.cpu(), m, r, g, None, *got)


def test_backward_against_differences():
    """dx and dgamma against central differences of the 64-bit forward."""
    R, C, h = 2, 24, 1e-6
    x, g, b = (t.double() for t in _case(R, C, 41, torch.float32))
    dy = randn((R, C), 42, dtype=torch.float32).double()

    def loss(x, g):
        mu, rs = _stats(x)
        return ((x - mu) * rs * g + b).mul(dy).sum()

    mu, rs = _stats(x)
    dx, dg = torch.empty(R, C, device=DEV), torch.empty(C, device=DEV)
    w = ws(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C))
    f = lambda t: t.float().to(DEV)
    aqfq.aqfq_layernorm_bwd(f(dy), f(x), f(mu[:, 0]), f(rs[:, 0]), f(g), dx, dgamma=dg, workspace=w)
    num = torch.empty_like(x)
    for i in range(R):
        for j in range(C):
            e = torch.zeros_like(x)
            e[i, j] = h
            num[i, j] = (loss(x + e, g) - loss(x - e, g)) / (2 * h)
    # differences: h^2 third derivatives and 2^-52 |loss| / h; kernel: 100 U of terms of order 10
    close(dx, num, torch.full_like(num, 1e-4))
    ng = torch.stack([(loss(x, g + h * torch.eye(C)[j]) - loss(x, g - h * torch.eye(C)[j])) / (2 * h)
                      for j in range(C)])
    close(dg, ng, torch.full_like(ng, 1e-4))


def test_empty_rows():
    e = torch.empty(0, 96, device=DEV)
    z = torch.empty(0, device=DEV)
    aqfq.aqfq_layernorm_fwd(e, None, None, EPS, e, mean=z, rstd=z)
    dg, db = torch.full((96,), 2.0, device=DEV), torch.full((96,), 2.0, device=DEV)
    w = ws(16)
    aqfq.aqfq_layernorm_bwd(e, e, z, z, None, e, dgamma=dg, dbeta=db, accumulate=True, workspace=w)
    assert bool((dg == 2).all()) and bool((db == 2).all())
    aqfq.aqfq_layernorm_bwd(e, e, z, z, None, e, dgamma=dg, dbeta=db, workspace=w)
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_offsets_beyond_32_bits():
    C, ld = 136, (1 << 32) + 64
    big = torch.empty(ld + C, dtype=torch.bfloat16, device=DEV)
    v = big.as_strided((2, C), (ld, 1))
    x, g, b = _case(2, C, 51, torch.bfloat16)
    v.copy_(x)
    m, r = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
    y = torch.empty(2, C, dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_layernorm_fwd(v, g.to(DEV), b.to(DEV), EPS, y, mean=m, rstd=r)
    torch.cuda.synchronize()
    _check_fwd(x, g, b, y, m, r)
    dx = torch.empty_like(y)
    aqfq.aqfq_layernorm_bwd(y, v, m, r, g.to(DEV), dx)
    torch.cuda.synchronize()
    _check_bwd(x, y.cpu(), m, r, g, None, dx, None, None)


def test_same_bits_again_and_on_another_stream():
    R, C = 2000, 1003
    x, g, b = _case(R, C, 61, torch.bfloat16)
    xd, gd, bd, dy = x.to(DEV), g.to(DEV), b.to(DEV), randn((R, C), 62).to(DEV)
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

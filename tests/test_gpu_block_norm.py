"""The norms, gate and residual between two blocks against 64-bit formulas.

Bounds (U the unit roundoff of binary32, D = C / 256 + 64 the depth of a sum over C columns, R + 64
over rows; hardware reciprocal square roots are within 4 U).
Forward: mean squares are sums of terms of one sign, (D + 3) U of themselves off, a reciprocal root
half of that and 6 U.  n takes five roundings, h one more; h's error e enters rstd_pre as
mean(|h| e) / mean(h^2).  Backward, from the stored h and the call's own rstd: with A = |rstd u| + |dh|,
B = A + |m2 hh|, m2 = rstd mean(u hh): each product adds one or two roundings of its factors,
the means D; m2 is then (D + 6) U rstd mean|u hh| off, dx 4 U B + that |hh|, and mean(c dx fh) the sum of
(D + 8) U of mean(|c fh| A) and |m2| mean|c fh hh|, and m2's error times the latter.  A BF16 value is
rounded by at most 2^-8 of itself at the end."""
import pytest
import torch

from layerlib import BF, DEV, Framed, U, close, randn, ws
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 8), (64, 100), (2, 255), (300, 256), (33, 1003), (7, 2056),
          (1000, 768), (701, 512), (5, 5000), (3, 8192), (2, 20000), (160, 9001),
          # rows that allow accesses of two elements only
          (300, 6), (333, 250), (77, 510), (40, 1018), (3, 2002), (160, 4090), (155, 8190)]
EPS = 1e-6


def inputs(R, C, seed, dtype, pdtype):
    x = randn((R, C), seed, 2.0, torch.float32)
    x[:, ::61] *= 20.0
    f = randn((R, C), seed + 1, 0.7, torch.float32) * torch.logspace(-2, 2, R)[:, None]
    v = [1 + randn((C,), seed + 2, 0.2, torch.float32), randn((C,), seed + 3, 0.5, torch.float32),
         1 + randn((C,), seed + 4, 0.2, torch.float32)]
    return x.to(dtype), f.to(dtype), *(t.to(pdtype) for t in v)


def ones(C):
    return torch.ones(C).double()


def forward64(x, f, post, gpost, gate, alpha, gpre, eps, C):
    """(value, bound before the last rounding) of h, y, rstd_post, rstd_pre."""
    D = C / 256 + 64
    out = {}
    c = alpha * (ones(C) if gate is None else gate.double())
    c = c * (ones(C) if gpost is None else gpost.double())
    h = 0.0 if x is None else x.double()
    eh = 0.0
    if f is not None:
        n = f.double()
        en = 0.0
        if post:
            r = 1 / torch.sqrt((n * n).mean(1, keepdim=True) + eps)
            er = (D / 2 + 8) * U
            out["rstd_post"] = (r[:, 0], er * r[:, 0])
            n, en = n * r, er
        h = h + c * n
        eh = (en + 5 * U) * (c * n).abs()
    eh = eh + U * h.abs() if f is not None else torch.zeros_like(h)
    out["h"] = (h, eh)
    ms = (h * h).mean(1, keepdim=True)
    r = 1 / torch.sqrt(ms + eps)
    er = (D / 2 + 8) * U + (h.abs() * eh).mean(1, keepdim=True) / (ms + eps)
    out["rstd_pre"] = (r[:, 0], (er * r)[:, 0])
    g = ones(C) if gpre is None else gpre.double()
    out["y"] = (h * r * g, eh * r * g.abs() + (er + 3 * U) * (h * r * g).abs())
    return out


def check(got, ref, dtype, what):
    want, tol = ref
    if dtype == torch.bfloat16:
        tol = tol + BF * (want.abs() + tol)
    close(got, want, tol, what)


LAYOUTS = ((0, 0), (8, 8), (3, 1), (2, 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post", [True, False])
def test_forward(dtype, pdtype, post):
    for i, (R, C) in enumerate(SHAPES):
        x, f, gpost, gate, gpre = inputs(R, C, 10 * i, dtype, pdtype)
        gpost = gpost if post and i % 3 else None
        gate = gate if i % 4 else None
        for pad, off in LAYOUTS:
            fx, ff = Framed(R, C, dtype, pad, off, x), Framed(R, C, dtype, pad, off, f)
            fh, fy = Framed(R, C, dtype, pad, off), Framed(R, C, dtype, pad, off)
            rp, rq = (torch.full((R,), -1.0, device=DEV) for _ in range(2))
            d = lambda t: None if t is None else t.to(DEV)
            aqfq.aqfq_block_norm_fwd(fx.view, ff.view, EPS, h=fh.view, y=fy.view, post=post, gamma_post=d(gpost),
                                     gate=d(gate), alpha=0.5, gamma_pre=d(gpre), rstd_pre=rq,
                                     rstd_post=rp if post else None)
            torch.cuda.synchronize()
            ref = forward64(x, f, post, gpost, gate, 0.5, gpre, EPS, C)
            check(fh.view, ref["h"], dtype, f"h {R}x{C}")
            check(fy.view, ref["y"], dtype, f"y {R}x{C}")
            check(rq, ref["rstd_pre"], None, "rstd_pre")
            if post:
                check(rp, ref["rstd_post"], None, "rstd_post")
            assert fh.intact() and fy.intact()


def bwd64(dy, dh, h, f, rp, rq, gpost, gate, alpha, gpre, R, C):
    """(value, bound) of the gradients from the forward's stored h and its rstd (rp, rq)."""
    D, out = C / 256 + 64, {}
    mean = lambda t: t.mean(1, keepdim=True)
    z = torch.zeros(R, C).double()
    g = ones(C) if gpre is None else gpre.double()
    post = ones(C) if gpost is None else gpost.double()
    ga = ones(C) if gate is None else gate.double()
    c = alpha * ga * post
    rq = torch.zeros(R, 1).double() if rq is None else rq.double().cpu()[:, None]
    d = z if dy is None else dy.double()
    hh = z if dy is None else h.double() * rq
    e = z if dh is None else dh.double()
    u = d * g
    m2 = rq * mean(u * hh)
    A = (rq * u).abs() + e.abs()
    B = A + (m2 * hh).abs()
    em2 = (D + 6) * U * rq * mean((u * hh).abs())
    dx = rq * u - m2 * hh + e
    edx = 4 * U * B + em2 * hh.abs()
    out["dx"] = (dx, edx)
    out["dgamma_pre"] = ((d * hh).sum(0), (R + 64) * U * (d * hh).abs().sum(0))
    if f is None:
        return out
    r = torch.ones(R, 1).double() if rp is None else rp.double().cpu()[:, None]
    fh = f.double() * r
    S, eS = (dx * fh).sum(0), ((edx + 2 * U * dx.abs()) * fh.abs()).sum(0) + (R + 64) * U * (dx * fh).abs().sum(0)
    for name, k in (("dgate", alpha * post), ("dgamma_post", alpha * ga)):
        out[name] = (k * S, k.abs() * (eS + 3 * U * S.abs()))
    v = c * dx
    ev = c.abs() * (edx + 3 * U * dx.abs())
    if rp is not None:
        m3 = mean(v * fh)
        cf = (c * fh).abs()
        em3 = ((D + 8) * U * (mean(cf * A) + m2.abs() * mean(cf * hh.abs())) + em2 * mean(cf * hh.abs())
               + 2 * U * m3.abs())
        df = r * (v - fh * m3)
        out["df"] = (df, r * (ev + em3 * fh.abs() + 3 * U * (fh * m3).abs()) + 2 * U * df.abs())
    else:
        out["df"] = (v, ev)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post", [True, False])
def test_backward(dtype, pdtype, post):
    for i, (R, C) in enumerate(SHAPES):
        x, f, gpost, gate, gpre = inputs(R, C, 10 * i, dtype, pdtype)
        gpost = gpost if post and i % 3 else None
        gate = gate if i % 4 else None
        gpre = gpre if i % 5 else None
        # plain rstd of the stored values, as a forward gives them
        ref = forward64(x, f, post, gpost, gate, 0.5, gpre, EPS, C)
        h = ref["h"][0].to(dtype)
        rq = ref["rstd_pre"][0].float().to(DEV)
        rp = ref["rstd_post"][0].float().to(DEV) if post else None
        dy, dh = (randn((R, C), 900 + i + k, dtype=torch.float32).to(dtype) for k in (0, 40))
        if i % 6 == 4:
            dh = None
        if i % 7 == 5:
            dy = gpre = None
        base = randn((3, C), 77 + i, 3.0, torch.float32)
        pad, off = LAYOUTS[i % 4]
        for acc in (False, True):
            fr = {n: None if t is None else Framed(R, C, dtype, pad, off, t)
                  for n, t in (("dy", dy), ("dh", dh), ("h", h), ("f", f))}
            fx, fd = Framed(R, C, dtype, pad, off), Framed(R, C, dtype, pad, off)
            vec = base.to(DEV).clone() if acc else torch.full((3, C), float("nan"), device=DEV)
            d = lambda t: None if t is None else t.to(DEV)
            view = lambda n: None if fr[n] is None else fr[n].view
            kw = {"dgate": vec[0], "dgamma_post": vec[1] if post else None,
                  "dgamma_pre": vec[2] if dy is not None else None}
            aqfq.aqfq_block_norm_bwd(view("dy"), view("dh"), view("h"), view("f"), rstd_post=rp,
                                     rstd_pre=rq if dy is not None else None, gamma_post=d(gpost), gate=d(gate),
                                     alpha=0.5, gamma_pre=d(gpre), dx=fx.view, df=fd.view, accumulate=acc,
                                     workspace=ws(aqfq.aqfq_block_norm_bwd_workspace_bytes(R, C)), **kw)
            torch.cuda.synchronize()
            want = bwd64(dy, dh, h, f, rp, rq, gpost, gate, 0.5, gpre, R, C)
            check(fx.view, want["dx"], dtype, f"dx {R}x{C}")
            check(fd.view, want["df"], dtype, f"df {R}x{C}")
            for k, n in enumerate(("dgate", "dgamma_post", "dgamma_pre")):
                if kw[n] is not None:
                    v, t = want[n]
                    if acc:
                        v, t = v + base[k].double(), t + U * (v + base[k].double()).abs()
                    check(vec[k], (v, t), None, f"{n} {R}x{C}")
            assert fx.intact() and fd.intact()


# rows that the rings of shared memory serve: every number of warps per row, full and ragged
# columns, a last stage with one row
RINGS = [(2435, 4096, torch.bfloat16), (2433, 2600, torch.bfloat16), (4867, 2048, torch.bfloat16),
         (4865, 1032, torch.bfloat16), (1217, 8192, torch.bfloat16), (1219, 4104, torch.bfloat16),
         (1218, 4096, torch.float32), (4867, 1048, torch.float32), (613, 8192, torch.float32)]
RINGS_BACK = [(1217, 4096, torch.bfloat16), (1220, 2056, torch.bfloat16), (2433, 2048, torch.bfloat16),
              (1219, 1032, torch.bfloat16), (609, 8192, torch.bfloat16), (610, 4104, torch.bfloat16),
              (1219, 2048, torch.float32), (611, 4096, torch.float32)]
# many rows in registers, several groups of warps per block
MANY_BACK = [(4865, 1024, torch.bfloat16), (4871, 520, torch.bfloat16), (9731, 512, torch.bfloat16),
             (9729, 264, torch.bfloat16), (4867, 512, torch.float32), (2440, 1024, torch.float32),
             (2000, 1003, torch.bfloat16), (3001, 333, torch.float32), (700, 4001, torch.bfloat16), (333, 5001, torch.bfloat16),
             (157, 8191, torch.float32), (2000, 1002, torch.bfloat16), (3001, 334, torch.float32),
             (700, 4002, torch.bfloat16), (333, 5002, torch.bfloat16)]


@pytest.mark.parametrize("R,C,dtype", RINGS)
def test_forward_from_a_ring(R, C, dtype):
    G = aqfq.aqfq_selftest_block_norm_ring(False, dtype, R, C)
    assert G == (4 if C <= 2048 else 8 if C <= 4096 else 16)
    x, f, gpost, gate, gpre = inputs(R, C, 21, dtype, torch.bfloat16)
    for post in (True, False):
        fx, ff = Framed(R, C, dtype, 8, 8, x), Framed(R, C, dtype, 0, 0, f)
        fh, fy = Framed(R, C, dtype, 16, 8), Framed(R, C, dtype, 0, 0)
        rp, rq = (torch.full((R,), -1.0, device=DEV) for _ in range(2))
        gp = gpost if post else None
        kw = dict(post=post, gamma_post=None if gp is None else gp.to(DEV), gate=gate.to(DEV), alpha=0.5,
                  gamma_pre=gpre.to(DEV), rstd_post=rp if post else None)
        aqfq.aqfq_block_norm_fwd(fx.view, ff.view, EPS, h=fh.view, y=fy.view, rstd_pre=rq, **kw)
        only = torch.empty(R, C, dtype=dtype, device=DEV)
        aqfq.aqfq_block_norm_fwd(fx.view, ff.view, EPS, y=only, **kw)
        torch.cuda.synchronize()
        ref = forward64(x, f, post, gp, gate, 0.5, gpre, EPS, C)
        check(fh.view, ref["h"], dtype, f"h {R}x{C}")
        check(fy.view, ref["y"], dtype, f"y {R}x{C}")
        check(rq, ref["rstd_pre"], None, "rstd_pre")
        if post:
            check(rp, ref["rstd_post"], None, "rstd_post")
        assert fh.intact() and fy.intact() and torch.equal(only, fy.view)


@pytest.mark.parametrize("R,C,dtype", RINGS_BACK + MANY_BACK)
@pytest.mark.parametrize("post", [True, False])
def test_backward_of_many_rows(R, C, dtype, post):
    x, f, gpost, gate, gpre = inputs(R, C, 31, dtype, torch.float32)
    gpost = gpost if post else None
    ref = forward64(x, f, post, gpost, gate, 0.5, gpre, EPS, C)
    h = ref["h"][0].to(dtype)
    rq = ref["rstd_pre"][0].float().to(DEV)
    rp = ref["rstd_post"][0].float().to(DEV) if post else None
    dy, dh0 = (randn((R, C), 900 + k, dtype=torch.float32).to(dtype) for k in (0, 40))
    for dh in (dh0, None):
        G = aqfq.aqfq_selftest_block_norm_ring(True, dtype, R, C, dh is not None)
        assert G == (0 if (R, C, dtype) in MANY_BACK else 8 if C <= 2048 else 16)
        fr = {n: None if t is None else Framed(R, C, dtype, 8 * k, 8, t)
              for k, (n, t) in enumerate((("dy", dy), ("dh", dh), ("h", h), ("f", f)))}
        fx, fd = Framed(R, C, dtype, 8, 8), Framed(R, C, dtype, 0, 0)
        vec = torch.full((3, C), float("nan"), device=DEV)
        view = lambda n: None if fr[n] is None else fr[n].view
        aqfq.aqfq_block_norm_bwd(view("dy"), view("dh"), view("h"), view("f"), rstd_post=rp, rstd_pre=rq,
                                 gamma_post=None if gpost is None else gpost.to(DEV), gate=gate.to(DEV), alpha=0.5,
                                 gamma_pre=gpre.to(DEV), dx=fx.view, df=fd.view, dgate=vec[0],
                                 dgamma_post=vec[1] if post else None, dgamma_pre=vec[2],
                                 workspace=ws(aqfq.aqfq_block_norm_bwd_workspace_bytes(R, C)))
        torch.cuda.synchronize()
        want = bwd64(dy, dh, h, f, rp, rq, gpost, gate, 0.5, gpre, R, C)
        check(fx.view, want["dx"], dtype, f"dx {R}x{C}")
        check(fd.view, want["df"], dtype, f"df {R}x{C}")
        for k, n in enumerate(("dgate", "dgamma_post", "dgamma_pre")):
            if n != "dgamma_post" or post:
                check(vec[k], want[n], None, f"{n} {R}x{C}")
        assert fx.intact() and fd.intact()


def test_parts_of_the_call():
    """Without a residual, without a block (a plain norm), h or y alone; the same bits as together."""
    R, C = 9, 640
    x, f, gpost, gate, gpre = (t.to(DEV) for t in inputs(R, C, 3, torch.bfloat16, torch.float32))
    new = lambda: torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
    h, y, h2, y2 = new(), new(), new(), new()
    kw = dict(post=True, gamma_post=gpost, gate=gate, alpha=0.25)
    aqfq.aqfq_block_norm_fwd(x, f, EPS, h=h, y=y, gamma_pre=gpre, **kw)
    aqfq.aqfq_block_norm_fwd(x, f, EPS, h=h2, **kw)
    aqfq.aqfq_block_norm_fwd(x, f, EPS, y=y2, gamma_pre=gpre, **kw)
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2)
    c = lambda t: t.cpu()
    aqfq.aqfq_block_norm_fwd(x, None, EPS, y=y, gamma_pre=gpre)
    torch.cuda.synchronize()
    check(y, forward64(c(x), None, False, None, None, 1.0, c(gpre), EPS, C)["y"], torch.bfloat16, "plain norm")
    aqfq.aqfq_block_norm_fwd(None, f, EPS, h=h, y=y, gamma_pre=gpre, **kw)
    torch.cuda.synchronize()
    ref = forward64(None, c(f), True, c(gpost), c(gate), 0.25, c(gpre), EPS, C)
    check(h, ref["h"], torch.bfloat16, "h without x")
    check(y, ref["y"], torch.bfloat16, "y without x")
    # the gradient of the plain norm
    r = torch.empty(R, device=DEV)
    dy, dg, dx = f, torch.empty(C, device=DEV), new()
    aqfq.aqfq_block_norm_fwd(x, None, EPS, y=y, gamma_pre=gpre, rstd_pre=r)
    aqfq.aqfq_block_norm_bwd(dy, None, x, None, rstd_pre=r, gamma_pre=gpre, dx=dx, dgamma_pre=dg,
                             workspace=ws(aqfq.aqfq_block_norm_bwd_workspace_bytes(R, C)))
    torch.cuda.synchronize()
    want = bwd64(c(dy), None, c(x), None, None, c(r), None, None, 1.0, c(gpre), R, C)
    check(dx, want["dx"], torch.bfloat16, "dx of a plain norm")
    check(dg, want["dgamma_pre"], None, "dgamma_pre of a plain norm")


def test_gradients_against_differences():
    """The loss <y, wy> + <h, wh> in binary32 for steps along random directions."""
    R, C = 6, 96
    x, f, gpost, gate, gpre = (t.to(DEV).double() for t in inputs(R, C, 8, torch.float32, torch.float32))
    wy, wh = (randn((R, C), s, dtype=torch.float32).to(DEV) for s in (1, 2))

    def loss(x, f, gpost, gate, gpre):
        n = f / torch.sqrt((f * f).mean(1, keepdim=True) + EPS) * gpost
        h = x + 0.7 * gate * n
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * gpre
        return float((y * wy.double()).sum() + (h * wh.double()).sum())

    args = [x, f, gpost, gate, gpre]
    s = [t.float() for t in args]
    h, y, dx, df = (torch.empty(R, C, device=DEV) for _ in range(4))
    rp, rq = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    v = torch.empty(3, C, device=DEV)
    aqfq.aqfq_block_norm_fwd(s[0], s[1], EPS, h=h, y=y, post=True, gamma_post=s[2], gate=s[3], alpha=0.7,
                             gamma_pre=s[4], rstd_post=rp, rstd_pre=rq)
    aqfq.aqfq_block_norm_bwd(wy, wh, h, s[1], rstd_post=rp, rstd_pre=rq, gamma_post=s[2], gate=s[3], alpha=0.7,
                             gamma_pre=s[4], dx=dx, df=df, dgamma_post=v[0], dgate=v[1], dgamma_pre=v[2],
                             workspace=ws(aqfq.aqfq_block_norm_bwd_workspace_bytes(R, C)))
    torch.cuda.synchronize()
    for i, grad in enumerate((dx, df, v[0], v[1], v[2])):
        d = torch.randn(grad.shape, generator=torch.Generator().manual_seed(i)).double().to(DEV)
        # small beside every row: f's rows differ by 10^4, and a difference is off by the square
        # of the step over the row's size (at 1e-4 of the mean of all of them, by 0.1 in the
        # smallest row); in 64 bits its rounding is then below 1e-9 of `size`
        step = 1e-4 * float(args[i].abs().mean(-1).min())
        hi, lo = ([a + k * step * d if j == i else a for j, a in enumerate(args)] for k in (1, -1))
        num = (loss(*hi) - loss(*lo)) / (2 * step)
        ana = float((grad.double() * d).sum())
        size = float((grad.double() * d).abs().sum())
        # the third derivative times step^2, and binary32 gradients
        assert abs(num - ana) <= 1e-5 * size, i


def test_non_finite_rows_stay_alone_and_zero_rows():
    R, C = 6, 1000
    x, f, gpost, gate, gpre = inputs(R, C, 5, torch.float32, torch.float32)
    x[1, 3], f[3, 999], x[4], f[4] = float("nan"), float("inf"), 0.0, 0.0
    d = lambda t: t.to(DEV)
    h, y, dx, df = (torch.empty(R, C, device=DEV) for _ in range(4))
    rp, rq = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    kw = dict(gamma_post=d(gpost), gate=d(gate), alpha=0.5, gamma_pre=d(gpre), rstd_post=rp, rstd_pre=rq)
    aqfq.aqfq_block_norm_fwd(d(x), d(f), EPS, h=h, y=y, post=True, **kw)
    dy, dh = (d(randn((R, C), s, dtype=torch.float32)) for s in (6, 7))
    aqfq.aqfq_block_norm_bwd(dy, dh, h, d(f), dx=dx, df=df, **kw)
    torch.cuda.synchronize()
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(dx[1]).all())
    assert bool(torch.isnan(h[3, 999])) and bool(torch.isnan(y[3]).all())
    rows = torch.tensor([0, 2, 4, 5])
    for t in (h, y, dx, df):
        assert bool(torch.isfinite(t.cpu()[rows]).all())
    assert bool((h[4] == 0).all()) and bool((y[4] == 0).all())
    ref = forward64(x[rows], f[rows], True, gpost, gate, 0.5, gpre, EPS, C)
    check(y.cpu()[rows], ref["y"], None, "y")


def test_no_rows():
    C = 40
    e = torch.empty(0, C, device=DEV)
    v = torch.ones(3, C, device=DEV)
    aqfq.aqfq_block_norm_fwd(e, e, EPS, h=e, y=e)
    none = torch.empty(0, device=DEV)
    kw = dict(rstd_post=none, rstd_pre=none, dx=e, df=e, dgamma_post=v[0], dgate=v[1], dgamma_pre=v[2])
    aqfq.aqfq_block_norm_bwd(e, e, e, e, accumulate=True, **kw)
    torch.cuda.synchronize()
    assert bool((v == 1).all())
    aqfq.aqfq_block_norm_bwd(e, e, e, e, **kw)
    torch.cuda.synchronize()
    assert bool((v == 0).all())


@pytest.mark.parametrize("R,C", [(1, 2048), (37, 1003), (5000, 512)])
def test_captured_and_on_another_stream(R, C):
    x, f, gpost, gate, gpre = (t.to(DEV) for t in inputs(R, C, 4, torch.bfloat16, torch.bfloat16))
    out = []

    def run(o, stream=None):
        kw = dict(gamma_post=gpost, gate=gate, alpha=0.5, gamma_pre=gpre, rstd_post=o[4], rstd_pre=o[5],
                  stream=stream)
        aqfq.aqfq_block_norm_fwd(x, f, EPS, h=o[0], y=o[1], post=True, **kw)
        aqfq.aqfq_block_norm_bwd(o[1], o[0], o[0], f, dx=o[2], df=o[3], dgamma_post=o[6], dgate=o[7],
                                 dgamma_pre=o[8], workspace=o[9], **kw)

    for _ in range(3):
        out.append([torch.zeros(R, C, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
                   + [torch.zeros(n, device=DEV) for n in (R, R, C, C, C)]
                   + [ws(aqfq.aqfq_block_norm_bwd_workspace_bytes(R, C))])
    run(out[0])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    run(out[1], stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out[2])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for o in out[1:]:
        assert all(torch.equal(p, q) for p, q in zip(out[0][:9], o[:9]))


def test_offsets_beyond_32_bits():
    """Rows 2^22 elements apart, 1300 of them: the last start beyond 2^33 bytes and 2^32
    elements.  The results of packed rows, which the other tests hold to the formulas."""
    R, ld, dt = 1300, 1 << 22, torch.bfloat16
    whole = torch.empty(R * ld, dtype=dt, device=DEV)
    for C in (2048, 512, 250, 251, 9001):
        names = ("x", "f", "dy", "dh", "h", "y", "dx", "df")
        far = {n: whole.as_strided((R, C), (ld, 1), 16384 * k) for k, n in enumerate(names)}
        near = {n: randn((R, C), 900 + k, 1.0, dt).to(DEV) for k, n in enumerate(names)}
        for n in names:
            far[n].copy_(near[n])
        g = randn((C,), 950, 1.0, torch.float32).to(DEV)
        out = []
        for t in (far, near):
            rp, rq = (torch.empty(R, device=DEV) for _ in range(2))
            sums = torch.empty(3, C, device=DEV)
            ws = torch.empty(aqfq.aqfq_block_norm_bwd_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
            aqfq.aqfq_block_norm_fwd(t["x"], t["f"], EPS, h=t["h"], y=t["y"], post=True, gamma_post=g, gate=g,
                                     alpha=0.5, gamma_pre=g, rstd_post=rp, rstd_pre=rq)
            aqfq.aqfq_block_norm_bwd(t["dy"], t["dh"], t["h"], t["f"], rstd_post=rp, rstd_pre=rq, gamma_post=g,
                                     gate=g, alpha=0.5, gamma_pre=g, dx=t["dx"], df=t["df"], dgamma_post=sums[0],
                                     dgate=sums[1], dgamma_pre=sums[2], workspace=ws)
            out.append((rp, rq, sums))
        torch.cuda.synchronize()
        for a, b in zip(*out):
            assert torch.equal(a, b), C
        for n in ("h", "y", "dx", "df"):
            assert torch.equal(far[n], near[n]), (n, C)

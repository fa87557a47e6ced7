"""The gated feed-forward product and its gradient against 64-bit formulas, on every kernel that
a size may take.

Operands are small integers (times a power of two) where bits are compared: every sum is then
exact in any order, so the kept gate and up are met bit for bit, and a product of a smooth
activation (E of its value off, its derivative E of its two terms: test_gpu_activations.py) with
exact factors is one rounding per factor more.  A BF16 value is rounded by at most 2^-8 of itself
at the end.  General operands: sums as in test_gpu_linear.py."""
import numpy as np
import pytest
import torch

from layerlib import ACT_ERR, ACTS, BF, DEV, Framed, U, act64, close, grid_values, kept, new_ckpt, pack_ref, randn, ws
from learnable_scale_fake_gb300 import aqfq
from test_gpu_linear import ints, operand
from test_gpu_linear_paths import FORMS, product, slope, value

pytestmark = pytest.mark.gpu
# (M, N, K): one token to several tiles, ragged everywhere, N of every remainder
SIZES = [(1, 8, 8), (1, 128, 64), (1, 768, 2048), (2, 137, 1000), (7, 264, 520), (16, 1536, 768), (33, 127, 4104),
         (64, 256, 512), (65, 391, 72), (128, 128, 64), (129, 257, 128), (200, 1000, 40), (300, 520, 1032),
         (515, 776, 136), (1000, 1544, 264)]
IDS = ["x".join(map(str, s)) for s in SIZES]
NAMES = list(ACTS)


def run_fwd(x, w, act, fmt=None, group=0, seed=0):
    M, K = x.shape
    N = w.shape[0] // 2
    fx, fw = operand(x, seed), operand(w, seed + 1)
    fy = Framed(M, N, torch.bfloat16, seed % 3, seed % 2)
    kw, parts = {}, []
    if fmt:
        for n in ("gate", "up"):
            ck, codes, scale = new_ckpt(M, N, fmt, group)
            kw[n] = ck
            parts.append((codes, scale))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    aqfq.aqfq_gated_fwd(fx.view, fw.view, fy.view, act=ACTS[act], error_flag=err,
                        workspace=ws(aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_FWD, M, N, K)), **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and fy.intact() and fx.intact() and fw.intact()
    return fy.view, parts


def check_fwd(M, N, K, act, form, seed=0, div=8.0):
    x, w = ints((M, K), 1 + seed, 1), ints((2 * N, K), 2 + seed, 1) / div
    fmt, group = form or (None, 0)
    y, parts = run_fwd(x, w, act, fmt, group, seed)
    p = product(x, w)
    g, u = p[:, :N], p[:, N:]
    a, e = value(g, act)
    ref = a * u.double()
    close(y, ref, e * u.abs() + (2 * U + BF) * ref.abs(), f"{act} {M}x{N}x{K}")
    for (codes, scale), t in zip(parts, (g, u)):
        q, s = pack_ref(t, fmt, group)
        np.testing.assert_array_equal(scale.cpu().numpy(), s)
        np.testing.assert_array_equal(grid_values(codes, fmt), q)


def two_ckpt(M, K, fmt, group, seed):
    out = []
    for i in range(2):
        ck, codes, scale = new_ckpt(M, K, fmt, group)
        aqfq.aqfq_ckpt8_pack(ck, randn((M, K), seed + i, 1.5).to(DEV))
        out.append((ck, codes, scale))
    torch.cuda.synchronize()
    return out


def check_grad(s, dp, y, g, u, act, what):
    """s, g, u in 64 bits."""
    K = g.shape[1]
    a, ea = value(g, act)
    d, ed = slope(g, act)
    if dp is not None:
        r = 5 * U + (BF if dp.dtype == torch.bfloat16 else 0)
        ref = s * u * d
        close(dp[:, :K], ref, (s * u).abs() * ed + r * ref.abs(), f"dg {what}")
        ref = s * a
        close(dp[:, K:], ref, s.abs() * ea + r * ref.abs(), f"du {what}")
    if y is not None:
        ref = a * u
        r = 5 * U + (BF if y.dtype == torch.bfloat16 else 0)
        close(y, ref, u.abs() * ea + r * ref.abs(), f"y {what}")


def check_dgrad(M, N, K, act, form, seed=0, div=8.0, hidden=True, place=None):
    """place: (pad, offset) of dp and y; by the seed if None."""
    dy, w = ints((M, N), 5 + seed, 1), ints((N, K), 6 + seed, 1) / div
    (cg, *g), (cu, *u) = two_ckpt(M, K, *form, seed=8 + seed)
    fd, fw = operand(dy, seed), operand(w, seed + 1)
    po, py = (place, place) if place else ((seed % 3, seed % 2), ((seed + 1) % 3, seed % 2))
    fo, fy = Framed(M, 2 * K, torch.bfloat16, *po), Framed(M, K, torch.bfloat16, *py)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    aqfq.aqfq_gated_dgrad(fd.view, fw.view, fo.view, cg, cu, act=ACTS[act], y=fy.view if hidden else None,
                          workspace=ws(aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_DGRAD, M, N, K)), error_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and fo.intact() and fy.intact()
    check_grad(product(dy, w.T).double(), fo.view, fy.view if hidden else None, kept(*g, *form), kept(*u, *form), act,
               f"{act} {M}x{N}x{K}")


@pytest.mark.parametrize("size", SIZES, ids=IDS)
@pytest.mark.parametrize("form", [None] + FORMS)
def test_forward(size, form):
    i = SIZES.index(size)
    for k in range(2):
        check_fwd(*size, NAMES[(i + k) % 5], form, seed=i + k)


@pytest.mark.parametrize("size", SIZES, ids=IDS)
@pytest.mark.parametrize("form", FORMS)
def test_gradient(size, form):
    M, K, N = size  # columns and inner axis of any length
    i = SIZES.index(size)
    check_dgrad(M, N, K, NAMES[i % 5], form, seed=i, hidden=i % 3 > 0)


# more than 152 tiles of 128 x 128 outputs: whole aligned blocks, ragged ones, an odd number of tile rows
ON_PAIRS = [(2048, 1280, 264), (2050, 1288, 200), (2303, 1261, 136)]


@pytest.mark.parametrize("act", NAMES)
@pytest.mark.parametrize("form", [None] + FORMS)
def test_forward_on_pairs(act, form):
    for i, (M, N, K) in enumerate(ON_PAIRS):
        plan = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_GATED, M, N, K)
        assert plan == {"kernel": "pair", "splits": 1, "tail": 0, "tail_splits": 0}
        check_fwd(M, N, K, act, form, seed=i)


@pytest.mark.parametrize("size,kernel", [((1000, 1544, 264), "pair"), ((500, 1000, 136), "tile"),
                                         ((129, 9600, 72), "pair"), ((128, 9728, 136), "tile"),
                                         ((129, 65, 2048), "narrow pair"), ((512, 768, 2048), "narrow pair"),
                                         ((700, 1500, 712), "narrow pair"), ((1023, 1149, 1000), "narrow pair"),
                                         ((128, 768, 2048), "tile"), ((512, 768, 2056), "tile")])
def test_each_kernel_near_the_borders(size, kernel):
    """(Half tiles: 64 outputs, of which a group of 128 takes two: kept so, the small tiles serve them.)"""
    assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_GATED, *size)["kernel"] == kernel
    for i, form in enumerate([None] + FORMS):
        check_fwd(*size, NAMES[i], form, seed=i)


@pytest.mark.parametrize("act", NAMES)
@pytest.mark.parametrize("form", FORMS)
def test_gradient_on_pairs(act, form):
    for i, (M, K, N) in enumerate([(2048, 2560, 264), (2050, 2568, 200), (2303, 2509, 136)]):
        assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_DGRAD, M, N, K)["kernel"] == "pair"
        check_dgrad(M, N, K, act, form, seed=i)


@pytest.mark.parametrize("act", NAMES)
@pytest.mark.parametrize("place", [(0, 0), (8, 8), (24, 16), (4, 0)])
def test_gradient_stored_in_boxes(act, place):
    """Outputs that allow 16-byte rows go to memory in boxes of 32 x 32, ragged ones cut off (the last
    place does not allow them); nothing around them is written."""
    for i, (M, K, N) in enumerate([(2048, 2560, 200), (2050, 2568, 136), (2303, 2520, 72)]):
        assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_DGRAD, M, N, K)["kernel"] == "pair"
        check_dgrad(M, N, K, act, FORMS[i], seed=i, hidden=i != 1, place=place)


def tails():
    """Sizes whose last tiles a second launch splits, by the number of slices (host only)."""
    found = {}
    for nr in (5, 6, 7, 9):
        for nc in range(8, 40):
            for depth in (3840, 4864, 6656):
                p = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_GATED, nr * 256, nc * 128, depth)
                if p["tail"]:
                    found.setdefault(p["tail_splits"], (nr * 256, nc * 128, depth))
    return found


def test_last_tiles_split_by_a_second_launch():
    found = tails()
    assert len(found) >= 3
    for i, (cut, (M, N, K)) in enumerate(sorted(found.items())):
        check_fwd(M - 5, N - 11, K - 24, NAMES[i % 5], FORMS[i % 4], seed=i % 3, div=64.0)
        check_fwd(M, N, K, NAMES[(i + 3) % 5], None if i % 2 else FORMS[(i + 1) % 4], div=64.0)
    for i, (M, K, N) in enumerate([(1787, 2805, 3816), (1280, 4352, 4096), (1280, 5120, 6656)]):
        assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_DGRAD, M, N, K)["tail"] > 0
        check_dgrad(M, N, K, NAMES[i + 2], FORMS[i], seed=i, div=64.0, hidden=i != 1)


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
def test_through_scratch(act):
    """Sums in slices through scratch, the epilogue in a second kernel."""
    for i, (M, N, K) in enumerate([(70, 300, 33000), (3, 129, 32768)]):
        assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_GATED, M, N, K)["splits"] > 1
        assert aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_FWD, M, N, K) > 0
        check_fwd(M, N, K, act, FORMS[i], div=128.0, seed=i)
        check_fwd(M, N, K, act, None, div=128.0, seed=i)
        check_dgrad(M, K, N, act, FORMS[i + 1], div=128.0, seed=i)


@pytest.mark.parametrize("size", [(1, 768, 2048), (200, 1000, 40), (515, 776, 1032), (2050, 1288, 512)])
@pytest.mark.parametrize("act", NAMES)
def test_general_operands(size, act):
    M, N, K = size
    x, w = randn((M, K), 1), randn((2 * N, K), 2, K ** -0.5)
    y, _ = run_fwd(x, w, act)
    p = x.double() @ w.double().T
    e = 2 * K * U * (x.double().abs() @ w.double().abs().T)
    g, u, eg, eu = p[:, :N], p[:, N:], e[:, :N], e[:, N:]
    a = act64(g, act)
    ea = 1.2 * eg + (ACT_ERR * g.abs() if act in ("gelu", "gelu_tanh", "silu") else 0)
    ref = a * u
    close(y, ref, ea * u.abs() + (a.abs() + ea) * eu + (2 * U + BF) * ref.abs(), act)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", NAMES)
def test_elementwise_gradient(dtype, form, act):
    for i, (R, C) in enumerate([(1, 1), (3, 7), (5, 32), (33, 136), (257, 1111), (64, 2048), (2, 9000)]):
        dy = randn((R, C), 30 + i, dtype=torch.float32).to(dtype)
        (cg, *g), (cu, *u) = two_ckpt(R, C, *form, seed=40 + i)
        for pad, off in ((0, 0), (3, 1)):
            fd, fo = Framed(R, C, dtype, pad, off, dy), Framed(R, 2 * C, dtype, pad, off)
            fy = Framed(R, C, dtype, pad, off)
            aqfq.aqfq_ckpt8_gated_bwd(cg, cu, ACTS[act], fd.view, dp=fo.view, y=fy.view)
            torch.cuda.synchronize()
            check_grad(dy.double(), fo.view, fy.view, kept(*g, *form), kept(*u, *form), act, f"{R}x{C}")
            assert fo.intact() and fy.intact()
            # each output alone
            fo2, fy2 = Framed(R, 2 * C, dtype, pad, off), Framed(R, C, dtype, pad, off)
            aqfq.aqfq_ckpt8_gated_bwd(cg, cu, ACTS[act], fd.view, dp=fo2.view)
            aqfq.aqfq_ckpt8_gated_bwd(cg, cu, ACTS[act], None, y=fy2.view)
            torch.cuda.synchronize()
            assert torch.equal(fo.view, fo2.view) and torch.equal(fy.view, fy2.view)


def test_gradient_against_differences():
    """Central differences of sum(dy act(g) u) in 64 bits at the kept values."""
    R, C = 5, 96
    dy = randn((R, C), 1, dtype=torch.float32)
    for act in ("gelu", "gelu_tanh", "silu", "none"):
        (cg, *g), (cu, *u) = two_ckpt(R, C, "int8", 64, seed=3)
        dp = torch.empty(R, 2 * C, device=DEV)
        aqfq.aqfq_ckpt8_gated_bwd(cg, cu, ACTS[act], dy.to(DEV), dp=dp)
        torch.cuda.synchronize()
        g, u, h = kept(*g, "int8", 64), kept(*u, "int8", 64), 1e-5
        loss = lambda g, u: dy.double() * act64(g, act) * u
        size = (dy.double() * u).abs() + dy.double().abs()
        num = torch.cat([(loss(g + h, u) - loss(g - h, u)) / (2 * h), (loss(g, u + h) - loss(g, u - h)) / (2 * h)], 1)
        # h^2 / 6 of a third derivative below 3, binary32 rounding, ACT_ERR of the terms
        assert bool(((dp.double().cpu() - num).abs() <= 1e-5 * torch.cat([size, size * (1 + g.abs())], 1)).all()), act


def test_non_finite_values_stay_where_they_belong():
    """A NaN in a row of x is that row's; one in up's first weight row is that column's, although
    gate's last tile reads past its rows into up's."""
    M, N, K = 140, 40, 256
    x, w = randn((M, K), 1), randn((2 * N, K), 2, K ** -0.5)
    x[3, 7] = float("nan")
    y, _ = run_fwd(x, w, "silu")
    bad = torch.isnan(y.cpu())
    assert bool(bad[3].all()) and int(bad.sum()) == N
    x[3, 7] = 0.0
    w[N] = float("nan")
    for form in [None] + FORMS:
        fmt, group = form or (None, 0)
        y, parts = run_fwd(x, w, "silu", fmt, group)
        bad = torch.isnan(y.cpu())
        assert bool(bad[:, 0].all()) and int(bad.sum()) == M
        if form:
            (_, sg), (_, su) = parts
            assert bool(torch.isfinite(sg).all()) and bool(torch.isnan(su[:, 0]).all())
            assert bool(torch.isfinite(su[:, 1:]).all())


def test_nothing_to_sum_and_nothing_to_write():
    z = lambda r, c: torch.empty(r, c, dtype=torch.bfloat16, device=DEV)
    for fmt in (None, "int8"):
        y = torch.full((3, 40), float("nan"), dtype=torch.bfloat16, device=DEV)
        kw = {}
        if fmt:
            kw = {n: new_ckpt(3, 40, fmt, 32)[0] for n in ("gate", "up")}
        aqfq.aqfq_gated_fwd(z(3, 0), z(80, 0), y, **kw)
        torch.cuda.synchronize()
        assert bool((y == 0).all())
        for c in kw.values():
            assert bool((c.tensors[0] == 0).all()) and bool((c.tensors[1] == 0).all())
    aqfq.aqfq_gated_fwd(z(0, 16), z(80, 16), z(0, 40))
    aqfq.aqfq_gated_fwd(z(4, 16), z(0, 16), z(4, 0))
    (cg, *g), (cu, *u) = two_ckpt(5, 24, "int8", 32, seed=1)
    dp = torch.full((5, 48), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = torch.full((5, 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_gated_dgrad(z(5, 0), z(0, 24), dp, cg, cu, y=y)
    torch.cuda.synchronize()
    assert bool((dp == 0).all())
    check_grad(None, None, y, kept(*g, "int8", 32), kept(*u, "int8", 32), "silu", "y")


def test_two_streams_and_a_replayed_graph():
    """The same bits from calls that overlap on two streams and from a captured graph."""
    M, N, K = 515, 776, 1032
    x, w = randn((M, K), 1).to(DEV), randn((2 * N, K), 2, K ** -0.5).to(DEV)
    dz, w2 = randn((M, 520), 3).to(DEV), randn((520, N), 4, 0.05).to(DEV)

    def buffers():
        cks = [new_ckpt(M, N, "e4m3", 64) for _ in range(2)]
        new = lambda c: torch.zeros(M, c, dtype=torch.bfloat16, device=DEV)
        return cks, [new(N), new(2 * N), new(N)]

    def run(b, stream=None):
        (g, u), (y, dp, h) = b
        aqfq.aqfq_gated_fwd(x, w, y, gate=g[0], up=u[0], stream=stream)
        aqfq.aqfq_gated_dgrad(dz, w2, dp, g[0], u[0], y=h, stream=stream)

    assert aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_FWD, M, N, K) == 0
    assert aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_DGRAD, M, 520, N) == 0
    b = [buffers() for _ in range(4)]
    run(b[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st, c in zip(streams, b[1:3]):
        run(c, stream=st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(b[3])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for cks, outs in b[1:]:
        assert all(torch.equal(p, q) for p, q in zip(b[0][1], outs))
        for c, d in zip(b[0][0], cks):
            assert torch.equal(c[1], d[1]) and torch.equal(c[2], d[2])


@pytest.mark.parametrize("N,K", [(264, 512), (2000, 512), (8192, 256)])
def test_offsets_beyond_32_bits(N, K):
    """Rows 2^24 elements apart, 300 of them: the last start beyond 2^33 bytes and 2^32 elements.
    The results of packed rows, which the other tests hold to the formulas."""
    M, ld = 300, 1 << 24
    whole = torch.empty(M * ld, dtype=torch.bfloat16, device=DEV)
    widths = {"x": K, "y": N, "dz": 136, "dp": 2 * N, "hidden": N, "dy": N, "dp2": 2 * N, "hidden2": N}
    near = {n: randn((M, c), 60 + i, 1.0).to(DEV) for i, (n, c) in enumerate(widths.items())}
    far = {n: whole.as_strided((M, c), (ld, 1), 65536 * i) for i, (n, c) in enumerate(widths.items())}
    for n in widths:
        far[n].copy_(near[n])
    w, w2 = randn((2 * N, K), 70, K ** -0.5).to(DEV), randn((136, N), 71, 0.1).to(DEV)
    for t in (far, near):
        (g, *_), (u, *_) = new_ckpt(M, N, "int8", 64), new_ckpt(M, N, "int8", 64)
        aqfq.aqfq_gated_fwd(t["x"], w, t["y"], gate=g, up=u,
                            workspace=ws(aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_FWD, M, N, K)))
        aqfq.aqfq_gated_dgrad(t["dz"], w2, t["dp"], g, u, y=t["hidden"],
                              workspace=ws(aqfq.aqfq_gated_workspace_bytes(aqfq.LINEAR_DGRAD, M, 136, N)))
        aqfq.aqfq_ckpt8_gated_bwd(g, u, aqfq.ACT_SILU, t["dy"], dp=t["dp2"], y=t["hidden2"])
        torch.cuda.synchronize()
    for n in ("y", "dp", "hidden", "dp2", "hidden2"):
        assert torch.equal(far[n], near[n]), n


# rows, outputs and inner axes that fill nothing evenly; one to sixteen slices
FEW = [(1, 8, 8), (1, 1, 9), (1, 768, 2048), (2, 13, 15), (3, 2000, 31), (5, 7, 8200), (7, 8192, 264), (8, 136, 1000),
       (8, 264, 520), (9, 520, 1003), (13, 20000, 64), (15, 1001, 129), (16, 1536, 768), (16, 33, 4104)]


@pytest.mark.parametrize("size", FEW, ids=["x".join(map(str, s)) for s in FEW])
def test_few_rows(size):
    assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_GATED, *size)["kernel"] == "few rows"
    for i, act in enumerate(NAMES):
        check_fwd(*size, act, None, seed=i)


def test_what_few_rows_are():
    plan = lambda *s: aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_GATED, *s)
    assert plan(17, 768, 2048)["kernel"] == "tile" and plan(16, 768, 7)["kernel"] == "tile"
    assert {plan(1, n, k)["splits"] for n in (8, 768, 2048, 8192, 20000) for k in (32, 64, 768, 2048)} == {1, 2, 4, 8, 16}
    check_fwd(17, 768, 2048, "silu", None)
    check_fwd(16, 768, 7, "silu", None)


def test_few_rows_stay_apart():
    """A row or a column that is not finite leaves the others' bits alone; NaN behind the inner axis
    and behind the last row is not read into them."""
    M, N, K = 5, 100, 77
    framed = operand(randn((M, K), 1), 1), operand(randn((2 * N, K), 2, K ** -0.5), 1)
    for f in framed:
        f.whole[f.mask] = float("nan")
    x, w = (f.view for f in framed)
    y, z = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    aqfq.aqfq_gated_fwd(x, w, y)
    x[2] = float("inf")
    w[7, 3] = float("nan")
    w[N + 9, 76] = float("inf")
    aqfq.aqfq_gated_fwd(x, w, z)
    torch.cuda.synchronize()
    rows, cols = [0, 1, 3, 4], [c for c in range(N) if c not in (7, 9)]
    assert y.isfinite().all()
    assert torch.equal(y[rows][:, cols], z[rows][:, cols])
    assert not z[2].isfinite().any() and z[:, 7].isnan().all() and not z[:, 9].isfinite().any()

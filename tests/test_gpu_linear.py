"""The linear products against 64-bit formulas.

Exact cases: rows of A with a single one, or small integers whose sums stay
below 2^24, make every sum exact in any order, so the BF16 result is bit for bit
the reference's: they show a wrong index, tile edge or layout at once.
General inputs: each product of two BF16 values is exact in binary32, a sum of
K of them is at most 2 K U sum|a b| off (twice the unit roundoff, should the
adder truncate); the activation adds its slope (at most 1.2) times that, plus
ACT_ERR; a stored BF16 value one rounding more."""
import numpy as np
import pytest
import torch

from layerlib import (ACT_ERR, ACTS, BF, DEV, Framed, U, act64, close, dact64, grid_values, kept,
                      new_ckpt, pack_ref, randn, ws)
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu
# (M, N, K): one token to several tiles, ragged everywhere, inner sizes below and above a stage
SIZES = [(1, 8, 8), (1, 128, 64), (1, 4096, 2048), (2, 136, 1000), (7, 264, 520), (16, 1536, 768),
         (33, 128, 4104), (64, 256, 512), (65, 392, 72), (128, 128, 64), (129, 257, 128),
         (200, 1000, 40), (256, 256, 256), (300, 520, 1032), (515, 776, 136), (1000, 1536, 264)]
IDS = ["x".join(map(str, s)) for s in SIZES]


def up8(v):
    return (v + 7) // 8 * 8


def operand(src, seed):
    """A strided operand: leading dimension a multiple of 8, 16-byte aligned."""
    R, C = src.shape
    return Framed(R, C, torch.bfloat16, up8(C) - C + 8 * (seed % 3), 8 * (seed % 2), src)


def ints(shape, seed, lim=4):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-lim, lim + 1, shape, generator=g).to(torch.bfloat16)


def run_fwd(x, w, bias=None, act="none", res=None, fmt=None, group=0, seed=0):
    M, K = x.shape
    N = w.shape[0]
    fx, fw = operand(x, seed), operand(w, seed + 1)
    fy = Framed(M, N, torch.bfloat16, seed % 3, seed % 2)
    fr = None if res is None else Framed(M, N, torch.bfloat16, seed % 2, 0, res)
    ck, codes, scale = new_ckpt(M, N, fmt, group) if fmt else (None, None, None)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    wsp = ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_FWD, M, N, K))
    aqfq.aqfq_linear_fwd(fx.view, fw.view, fy.view, bias=None if bias is None else bias.to(DEV),
                         act=ACTS[act], residual=None if fr is None else fr.view, ckpt=ck,
                         workspace=wsp, error_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and fy.intact()
    return fy.view, codes, scale


def run_dgrad(dy, w, act="none", ck=None, res=None, seed=0):
    M, N = dy.shape
    K = w.shape[1]
    fd, fw = operand(dy, seed), operand(w, seed + 1)
    fo = Framed(M, K, torch.bfloat16, seed % 3, seed % 2)
    fr = None if res is None else Framed(M, K, torch.bfloat16, seed % 2, 0, res)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    wsp = ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_DGRAD, M, N, K))
    aqfq.aqfq_linear_dgrad(fd.view, fw.view, fo.view, act=ACTS[act], ckpt=ck,
                           residual=None if fr is None else fr.view, workspace=wsp, error_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and fo.intact()
    return fo.view


def run_wgrad(dy, x, dtype=torch.bfloat16, base=None, seed=0):
    M, N = dy.shape
    K = x.shape[1]
    fd, fx = operand(dy, seed), operand(x, seed + 1)
    fo = Framed(N, K, dtype, seed % 3, seed % 2, base)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    wsp = ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_WGRAD, M, N, K))
    aqfq.aqfq_linear_wgrad(fd.view, fx.view, fo.view, accumulate=base is not None, workspace=wsp,
                           error_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and fo.intact()
    return fo.view


@pytest.mark.parametrize("size", SIZES, ids=IDS)
def test_small_integers_are_exact(size):
    """Integers of at most 4: sums of at most 16 K < 2^24."""
    M, N, K = size
    x, w, dy = ints((M, K), 1), ints((N, K), 2), ints((M, N), 3)
    for seed in (0, 1, 2):
        y, _, _ = run_fwd(x, w, seed=seed)
        assert torch.equal(y.cpu(), (x.double() @ w.double().T).bfloat16()), "forward"
        dx = run_dgrad(dy, w, seed=seed)
        assert torch.equal(dx.cpu(), (dy.double() @ w.double()).bfloat16()), "input gradient"
        dw = run_wgrad(dy, x, torch.float32, seed=seed)
        assert torch.equal(dw.cpu(), (dy.double().T @ x.double()).float()), "weight gradient"


@pytest.mark.parametrize("size", SIZES[:6] + SIZES[9:13], ids=IDS[:6] + IDS[9:13])
def test_one_hot_rows_pick_weights(size):
    """A row with a one at column j gives W[:, j]; NaN in W elsewhere does not
    reach it only where the formula keeps it out, so W is finite here."""
    M, N, K = size
    w = randn((N, K), 5)
    j = torch.arange(M) % K
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    x[torch.arange(M), j] = 1.0
    y, _, _ = run_fwd(x, w)
    assert torch.equal(y.cpu(), w.T[j])


def _pre(x, w, bias):
    p = x.double() @ w.double().T + (0 if bias is None else bias.double())
    K = x.shape[1]
    e = 2 * K * U * (x.double().abs() @ w.double().abs().T) + 2 * U * p.abs()
    return p, e


@pytest.mark.parametrize("size", SIZES, ids=IDS)
@pytest.mark.parametrize("act", list(ACTS))
def test_forward_epilogue(size, act):
    M, N, K = size
    i = SIZES.index(size)
    x, w = randn((M, K), 10 + i), randn((N, K), 20 + i, 0.05)
    bias = None if i % 4 == 3 else randn((N,), 30 + i, dtype=torch.bfloat16 if i % 2 else torch.float32)
    res = randn((M, N), 40 + i) if i % 3 else None
    y, _, _ = run_fwd(x, w, bias, act, res, seed=i)
    p, e = _pre(x, w, bias)
    ref = act64(p, act)
    tol = 1.2 * e + (ACT_ERR * p.abs() if act in ("gelu", "gelu_tanh", "silu") else 0)
    if res is not None:
        ref = ref + res.double()
    close(y, ref, tol + BF * ref.abs(), act)


@pytest.mark.parametrize("size", SIZES, ids=IDS)
@pytest.mark.parametrize("fmt,group", [("int8", 128), ("e4m3", 64), ("int8", 32)])
def test_forward_checkpoint(size, fmt, group):
    """The pre-activation in 8 bits: exact for integer sums; in general the kept
    value is half a step off the pre-activation, which is itself e off."""
    M, N, K = size
    i = SIZES.index(size)
    x, w = ints((M, K), 50 + i), ints((N, K), 60 + i)
    bias = ints((N,), 70 + i)
    p = (x.double() @ w.double().T + bias.double()).float()
    y, codes, scale = run_fwd(x, w, bias, "gelu", fmt=fmt, group=group, seed=i)
    q, s = pack_ref(p, fmt, group)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)
    np.testing.assert_array_equal(grid_values(codes, fmt), q)
    x, w = randn((M, K), 80 + i), randn((N, K), 90 + i, 0.05)
    _, codes, scale = run_fwd(x, w, None, "silu", fmt=fmt, group=group, seed=i)
    p, e = _pre(x, w, None)
    s = torch.from_numpy(scale.cpu().numpy()[:, np.arange(N) // group]).double()
    step = s if fmt == "int8" else torch.maximum(p.abs() * 2.0 ** -3, s * 2.0 ** -9)
    close(kept(codes, scale, fmt, group), p, 0.5 * step * (1 + 2.0 ** -10) + 2 * e + 4 * U * p.abs())
    n = scale.shape[1]
    pad = torch.zeros(M, n * group - N).double()
    amax = torch.cat([p.abs(), pad], 1).view(M, n, group).amax(2)
    emax = torch.cat([e, pad], 1).view(M, n, group).amax(2)
    qm = 127.0 if fmt == "int8" else 448.0
    close(scale * qm, amax, emax + 4 * U * amax)


@pytest.mark.parametrize("size", SIZES, ids=IDS)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_input_gradient_with_the_activation(size, act):
    M, N, K = size
    i = SIZES.index(size)
    fmt, group = [("int8", 128), ("e4m3", 32), ("int8", 64)][i % 3]
    dy, w = randn((M, N), 100 + i), randn((N, K), 110 + i, 0.05)
    ck, codes, scale = new_ckpt(M, K, fmt, group)
    aqfq.aqfq_ckpt8_pack(ck, randn((M, K), 120 + i, 1.5).to(DEV))
    res = randn((M, K), 130 + i) if i % 2 else None
    dx = run_dgrad(dy, w, act, ck if act != "none" or i % 2 else None, res, seed=i)
    p = kept(codes, scale, fmt, group)
    a, d = dy.double() @ w.double(), dact64(p, act)
    e = 2 * N * U * (dy.double().abs() @ w.double().abs())
    ref = a * d
    tol = 1.2 * e + (0 if act in ("none", "relu") else ACT_ERR * a.abs()) + 4 * U * ref.abs()
    if res is not None:
        ref = ref + res.double()
    close(dx, ref, tol + BF * ref.abs(), act)


@pytest.mark.parametrize("size", SIZES + [(2500, 136, 264), (5000, 768, 520)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient(size, dtype, accumulate):
    M, N, K = size
    i = M + N + K
    dy, x = randn((M, N), 140 + i), randn((M, K), 150 + i)
    base = randn((N, K), 160 + i, 3.0, dtype) if accumulate else None
    dw = run_wgrad(dy, x, dtype, base, seed=i % 3)
    ref = dy.double().T @ x.double()
    tol = 2 * M * U * (dy.double().abs().T @ x.double().abs())
    if base is not None:
        ref = ref + base.double()
    tol = tol + 2 * U * ref.abs() + (BF * ref.abs() if dtype == torch.bfloat16 else 0)
    close(dw, ref, tol)


def test_gradients_against_differences():
    """sum(dy * act(x W^T)) differentiated numerically in 64 bits along random
    directions of x and W, against the three calls chained as a layer's backward
    (forward with checkpoint, activation gradient, input and weight gradients).
    The 8-bit checkpoint is exact here: pre-activations are integers / 16 within
    +-120 / 16 whose group amax is 127 / 16."""
    M, N, K, h = 24, 128, 64, 1e-5
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-1, 2, (M, K), generator=g).bfloat16()
    w = (torch.randint(-2, 3, (N, K), generator=g) / 16.0).bfloat16()
    # the first column of every row carries the largest value of its group
    x[:, 0] = 1.0
    w[0] = 0.0
    w[0, 0] = 127.0 / 16.0
    w[1:, 0] = 0.0
    dy = randn((M, N), 6)
    y, codes, scale = run_fwd(x, w, None, "silu", fmt="int8", group=128)
    p = x.double() @ w.double().T
    assert torch.equal(kept(codes, scale, "int8", 128), p)
    ck = aqfq.ckpt8(aqfq.INT8, 128, codes, scale)
    dpre = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_ckpt8_act_bwd(ck, aqfq.ACT_SILU, dy.to(DEV), dx=dpre)
    dx, dw = run_dgrad(dpre.cpu(), w).cpu().double(), run_wgrad(dpre.cpu(), x, torch.float32).cpu().double()
    loss = lambda a, b: (act64(a @ b.T, "silu") * dy.double()).sum()
    X, W = x.double(), w.double()
    for s in range(4):
        vx, vw = torch.randn(M, K, generator=g).double(), torch.randn(N, K, generator=g).double()
        nx = (loss(X + h * vx, W) - loss(X - h * vx, W)) / (2 * h)
        nw = (loss(X, W + h * vw) - loss(X, W - h * vw)) / (2 * h)
        # dpre and dx are BF16: relative 2^-9 of every term of the inner products
        d = (dact64(p, "silu") * dy.double()).abs()
        bx = 2 * BF * ((d @ W.abs()) * vx.abs()).sum() + 1e-4
        bw = 2 * BF * ((d.T @ X.abs()) * vw.abs()).sum() + 1e-4
        assert abs((dx * vx).sum() - nx) <= bx and abs((dw * vw).sum() - nw) <= bw


def test_non_finite_rows_stay_alone():
    """A NaN in a row of x is seen in that row of y only; one in W in that column."""
    M, N, K = 200, 300, 136
    x, w = randn((M, K), 1), randn((N, K), 2)
    clean, _, _ = run_fwd(x, w, act="gelu")
    x[70, 5], w[133, 7] = float("nan"), float("inf")
    y, codes, scale = run_fwd(x, w, act="gelu", fmt="int8", group=32)
    ok = torch.ones(M, N, dtype=torch.bool)
    ok[70], ok[:, 133] = False, False
    assert bool(torch.isnan(y[70]).all())
    assert torch.equal(y.cpu()[ok], clean.cpu()[ok])
    assert bool(torch.isnan(scale[70]).all()) and bool(torch.isnan(scale[:, 133 // 32]).all())
    dw = run_wgrad(y.cpu(), x[:, :64].contiguous(), torch.float32)
    assert bool(torch.isfinite(dw.cpu()[torch.arange(N) != 133, 6:]).sum() == 0)


def test_empty_sizes():
    """No rows, no columns, an empty inner axis."""
    z = lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16)
    b = randn((40,), 1)
    res = randn((3, 40), 2)
    y, codes, scale = run_fwd(z(3, 0), z(40, 0), b, "relu", res, "int8", 32)
    p = b.double().expand(3, 40)
    ref = (torch.clamp(p, min=0) + res.double()).bfloat16()
    assert torch.equal(y.cpu(), ref)
    q, s = pack_ref(p.float().contiguous(), "int8", 32)
    np.testing.assert_array_equal(grid_values(codes, "int8"), q)
    assert bool((run_dgrad(z(5, 0), z(0, 24)) == 0).all())
    assert bool((run_wgrad(z(0, 16), z(0, 24)) == 0).all())
    base = randn((16, 24), 3, dtype=torch.float32)
    assert torch.equal(run_wgrad(z(0, 16), z(0, 24), torch.float32, base).cpu(), base)
    run_fwd(z(0, 16), z(24, 16))
    run_fwd(z(4, 16), z(0, 16))


def test_offsets_beyond_32_bits():
    """Rows of x and y more than 2^32 elements apart in total."""
    ld = (1 << 31) + 64
    big = torch.empty(2 * ld + 64, dtype=torch.bfloat16, device=DEV)
    xs = big.as_strided((3, 64), (ld, 1))
    x, w = ints((3, 64), 1), ints((136, 64), 2)
    xs.copy_(x)
    y = torch.empty(3, 136, dtype=torch.bfloat16, device=DEV)
    wsp = ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_FWD, 3, 136, 64))
    aqfq.aqfq_linear_fwd(xs, w.to(DEV), y, workspace=wsp)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), (x.double() @ w.double().T).bfloat16())
    ys = big.as_strided((3, 64), (ld, 1))
    aqfq.aqfq_linear_fwd(x.to(DEV), w[:64].contiguous().to(DEV), ys, workspace=wsp)
    torch.cuda.synchronize()
    assert torch.equal(ys.cpu(), (x.double() @ w[:64].double().T).bfloat16())


@pytest.mark.parametrize("size", [(1, 4096, 2048), (16, 1536, 768), (300, 520, 1032), (5000, 768, 520)])
def test_same_bits_again_and_on_another_stream(size):
    M, N, K = size
    x, w, dy = randn((M, K), 1).to(DEV), randn((N, K), 2).to(DEV), randn((M, N), 3).to(DEV)
    out = []
    for st in (None, torch.cuda.Stream(), None):
        y, dx = torch.empty_like(dy), torch.empty_like(x)
        dw = torch.empty(N, K, device=DEV)
        wsp = [ws(aqfq.aqfq_linear_workspace_bytes(k, M, N, K)) for k in range(3)]
        torch.cuda.synchronize()
        aqfq.aqfq_linear_fwd(x, w, y, act=aqfq.ACT_GELU, workspace=wsp[0], stream=st)
        aqfq.aqfq_linear_dgrad(dy, w, dx, workspace=wsp[1], stream=st)
        aqfq.aqfq_linear_wgrad(dy, x, dw, workspace=wsp[2], stream=st)
        torch.cuda.synchronize()
        out.append((y, dx, dw))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], o))


def test_many_tiles_exact():
    """More output tiles than the GPU has SMs, in all three products."""
    M, N, K = 2100, 2056, 200
    x, w, dy = ints((M, K), 1), ints((N, K), 2), ints((M, N), 3, 1)
    y, _, _ = run_fwd(x, w)
    assert torch.equal(y.cpu(), (x.float() @ w.float().T).bfloat16())
    dx = run_dgrad(dy, w)
    assert torch.equal(dx.cpu(), (dy.float() @ w.float()).bfloat16())
    x2, dy2 = ints((72, 2056), 4), ints((72, 2100), 5)
    dw = run_wgrad(dy2, x2, torch.float32)
    assert torch.equal(dw.cpu(), dy2.float().T @ x2.float())


@pytest.mark.parametrize("M,N", [(2560, 2056), (2550, 2300), (4608, 1290)])
def test_many_tiles_in_clusters_of_two_pairs_exact(M, N):
    """An even number of tile rows: two pairs share their columns' operand; full
    rounds, a ragged last round, ragged edges in both axes."""
    K = 328
    x, w, dy = ints((M, K), 1), ints((N, K), 2), ints((M, N), 3, 1)
    for seed in (0, 1):
        y, codes, scale = run_fwd(x, w, None, "none", None, "int8", 128, seed=seed)
        p = x.float() @ w.float().T
        assert torch.equal(y.cpu(), p.bfloat16())
        q, s = pack_ref(p, "int8", 128)
        np.testing.assert_array_equal(grid_values(codes, "int8"), q)
        dy2, w2 = ints((M, K), 4), ints((K, N), 5)
        dx = run_dgrad(dy2, w2, seed=seed)
        assert torch.equal(dx.cpu(), (dy2.float() @ w2.float()).bfloat16())
        dy3, x3 = ints((K, M), 6), ints((K, N), 7)
        dw = run_wgrad(dy3, x3, torch.float32, seed=seed)
        assert torch.equal(dw.cpu(), dy3.float().T @ x3.float())


def test_last_tiles_split_by_a_second_launch_exact():
    """A long inner axis whose last round has few tiles: those are split along it."""
    M, N, K = 2560, 2304, 4104  # 90 tiles
    x, w = ints((M, K), 1, 1), ints((N, K), 2, 1)
    bias, res = ints((N,), 3), ints((M, N), 4)
    y, codes, scale = run_fwd(x, w, bias, "relu", res, "e4m3", 64)
    p = (x.float().cuda() @ w.float().cuda().T).cpu() + bias.float()
    assert torch.equal(y.cpu(), (torch.clamp(p, min=0) + res.float()).bfloat16())
    q, s = pack_ref(p, "e4m3", 64)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)
    np.testing.assert_array_equal(grid_values(codes, "e4m3"), q)


@pytest.mark.parametrize("size", [(33000, 136, 264), (32800, 8, 520), (40000, 1536, 2056)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_inner_axis_through_scratch(size, accumulate):
    """Weight gradients of many tokens: the sum is cut into slices whose partial sums
    meet in scratch.  Entries -1, 0, 1 keep every sum exact in binary32."""
    M, N, K = size
    assert aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_WGRAD, M, N, K) > 0
    dy, x = ints((M, N), 1, 1), ints((M, K), 2, 1)
    base = ints((N, K), 3).float() if accumulate else None
    dw = run_wgrad(dy, x, torch.float32, base, seed=M % 3)
    ref = dy.float().to(DEV).T @ x.float().to(DEV)
    if accumulate:
        ref = ref + base.to(DEV)
    assert torch.equal(dw, ref)


def test_forward_with_a_long_inner_axis_through_scratch():
    """The finishing kernel's forward epilogue: bias, checkpoint, activation, residual."""
    M, N, K = 70, 300, 33000
    x, w = ints((M, K), 1, 1), ints((N, K), 2, 1)
    assert aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_FWD, M, N, K) > 0
    bias, res = ints((N,), 3), ints((M, N), 4)
    y, codes, scale = run_fwd(x, w, bias, "relu", res, "int8", 128)
    p = (x.float().to(DEV) @ w.float().to(DEV).T).cpu() + bias.float()
    assert torch.equal(y.cpu(), (torch.clamp(p, min=0) + res.float()).bfloat16())
    q, s = pack_ref(p, "int8", 128)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)
    np.testing.assert_array_equal(grid_values(codes, "int8"), q)
    ck, codes, scale = new_ckpt(M, N, "e4m3", 32)
    aqfq.aqfq_ckpt8_pack(ck, randn((M, N), 5).to(DEV))
    dy, w2 = ints((M, K), 6, 1), ints((K, N), 7, 1)
    dx = run_dgrad(dy, w2, "relu", ck)
    keep = (kept(codes, scale, "e4m3", 32) > 0).float()
    ref = (dy.float().to(DEV) @ w2.float().to(DEV)).cpu() * keep
    assert torch.equal(dx.cpu(), ref.bfloat16())


def test_workspace_is_checked_and_bounded():
    need = aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_WGRAD, 33000, 136, 264)
    dy, x = torch.zeros(33000, 136, device=DEV).bfloat16(), torch.zeros(33000, 264, device=DEV).bfloat16()
    dw = torch.empty(136, 264, device=DEV)
    for w in (None, ws(need - 16)):
        with pytest.raises(aqfq.AqfqError) as e:
            aqfq.aqfq_linear_wgrad(dy, x, dw, workspace=w)
        assert e.value.status == 5
    for M, N, K in ((1 << 20, 4096, 4096), (1 << 20, 264, 264), (1 << 22, 1536, 2048)):
        assert aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_WGRAD, M, N, K) <= 64 << 20


# 77 to 152 tiles of 128 x 128: one slice each, the sums go straight through the epilogue
@pytest.mark.parametrize("size", [(1000, 264, 1544), (1100, 136, 1290)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("fmt,group", [("int8", 32), ("e4m3", 128)])
def test_input_gradient_of_whole_sums(size, act, fmt, group):
    M, N, K = size
    i = group % 3
    dy, w = randn((M, N), 400 + i), randn((N, K), 410 + i, 0.05)
    ck, codes, scale = new_ckpt(M, K, fmt, group)
    aqfq.aqfq_ckpt8_pack(ck, randn((M, K), 420 + i, 1.5).to(DEV))
    res = randn((M, K), 430 + i) if i else None
    dx = run_dgrad(dy, w, act, ck, res, seed=i)
    a, d = dy.double() @ w.double(), dact64(kept(codes, scale, fmt, group), act)
    e = 2 * N * U * (dy.double().abs() @ w.double().abs())
    ref = a * d
    tol = 1.2 * e + (0 if act in ("none", "relu") else ACT_ERR * a.abs()) + 4 * U * ref.abs()
    if res is not None:
        ref = ref + res.double()
    close(dx, ref, tol + BF * ref.abs(), act)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_of_whole_sums(dtype, accumulate):
    M, N, K = 200, 1000, 1290
    dy, x = randn((M, N), 440), randn((M, K), 441)
    base = randn((N, K), 442, 3.0, dtype) if accumulate else None
    for seed in (0, 1, 2):
        dw = run_wgrad(dy, x, dtype, base, seed=seed)
        ref = dy.double().T @ x.double()
        tol = 2 * M * U * (dy.double().abs().T @ x.double().abs())
        if base is not None:
            ref = ref + base.double()
        tol = tol + 2 * U * ref.abs() + (BF * ref.abs() if dtype == torch.bfloat16 else 0)
        close(dw, ref, tol)


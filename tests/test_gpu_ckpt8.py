"""8-bit activation checkpoints against the definition: codes and scales bit for
bit (the quotient is the IEEE binary32 one), the recomputed activation, its
gradient and the bias gradient against 64-bit formulas.

Bounds: an activation's value is |x| (ACT_ERR) off and its derivative ACT_ERR,
a column sum of R terms (R + 64) U of the sum of their sizes; a stored BF16
value one rounding more."""
import numpy as np
import pytest
import torch

from layerlib import (ACT_ERR, ACTS, BF, DEV, FMTS, Framed, U, act64, close, dact64, grid_values,
                      kept, new_ckpt, pack_ref, randn, ws)
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 7), (3, 8), (2, 32), (5, 33), (17, 100), (4, 257), (33, 1000), (1, 4099),
          (700, 264), (9, 4096)]


def _x(R, C, seed, dtype=torch.float32):
    x = randn((R, C), seed, dtype=torch.float32)
    x[:, ::97] *= 30.0
    if C > 40:
        x[0, 32:64] = 0.0          # a group of zeros
        x[-1, -1] = 1e-30          # far below its group's step
    return x.to(dtype)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pack_is_the_definition_bit_for_bit(fmt, group, dtype):
    for i, (R, C) in enumerate(SHAPES):
        x = _x(R, C, 100 + i, dtype)
        for pad, off in ((0, 0), (3, 1)):
            f = Framed(R, C, dtype, pad, off, x)
            ck, codes, scale = new_ckpt(R, C, fmt, group)
            aqfq.aqfq_ckpt8_pack(ck, f.view)
            torch.cuda.synchronize()
            q, s = pack_ref(x, fmt, group)
            np.testing.assert_array_equal(scale.cpu().numpy(), s)
            np.testing.assert_array_equal(grid_values(codes, fmt), q, err_msg=f"{R}x{C} pad {pad}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_pack_at_rounding_midpoints_and_extreme_scales(fmt):
    """Quotients at and next to the grid's midpoints, groups from subnormal to
    the largest values, one whose scale underflows to zero."""
    rows = []
    for e in (-149, -140, -127, -100, -64, 0, 64, 100, 119):
        qmax = 127.0 if fmt == "int8" else 448.0
        s = 2.0 ** max(e, -149)
        mids = (np.arange(126) + 0.5 if fmt == "int8" else
                (np.unique(np.abs(np.nan_to_num(kept_grid(fmt))))[:-1]
                 + np.unique(np.abs(np.nan_to_num(kept_grid(fmt))))[1:]) / 2)
        v = np.resize(mids, 127) * s
        v[1::3] = np.nextafter(v[1::3].astype(np.float32), np.float32(np.inf))
        v[2::3] = np.nextafter(v[2::3].astype(np.float32), np.float32(0))
        rows.append(np.concatenate([[qmax * s], v]).astype(np.float32))
    rows.append(np.full(128, 2.0 ** -149, np.float32))  # amax / qmax is zero
    x = torch.from_numpy(np.stack(rows))
    x[:, ::2] *= -1
    ck, codes, scale = new_ckpt(*x.shape, fmt, 128)
    aqfq.aqfq_ckpt8_pack(ck, x.to(DEV))
    torch.cuda.synchronize()
    q, s = pack_ref(x, fmt, 128)
    np.testing.assert_array_equal(scale.cpu().numpy(), s)
    np.testing.assert_array_equal(grid_values(codes, fmt), q)


def kept_grid(fmt):
    return grid_values(torch.arange(256, dtype=torch.uint8), fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_non_finite_groups_come_back_nan_and_alone(fmt):
    x = _x(4, 200, 7)
    x[0, 5], x[1, 70], x[2, 199] = float("nan"), float("inf"), -float("inf")
    ck, codes, scale = new_ckpt(4, 200, fmt, 64)
    y = torch.empty(4, 200, device=DEV)
    aqfq.aqfq_ckpt8_pack(ck, x.to(DEV))
    aqfq.aqfq_ckpt8_unpack(ck, y)
    torch.cuda.synchronize()
    bad = torch.zeros(4, 200, dtype=torch.bool)
    bad[0, :64], bad[1, 64:128], bad[2, 192:] = True, True, True
    assert torch.equal(torch.isnan(y.cpu()), bad)
    assert int(codes.cpu()[bad].max()) == 0
    q, s = pack_ref(x, fmt, 64)
    np.testing.assert_array_equal(grid_values(codes, fmt)[~bad.numpy()], q[~bad.numpy()])


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unpack_recomputes_the_activation(act, dtype):
    for i, (R, C) in enumerate(SHAPES):
        fmt, group = ("int8", 32) if i % 2 else ("e4m3", 128)
        ck, codes, scale = new_ckpt(R, C, fmt, group)
        aqfq.aqfq_ckpt8_pack(ck, _x(R, C, 200 + i).to(DEV))
        f = Framed(R, C, dtype, 5, 3) if i % 3 == 0 else Framed(R, C, dtype)
        aqfq.aqfq_ckpt8_unpack(ck, f.view, act=ACTS[act])
        torch.cuda.synchronize()
        p = kept(codes, scale, fmt, group)
        ref = act64(p, act)
        tol = ACT_ERR * p.abs() if act in ("gelu", "gelu_tanh", "silu") else torch.zeros_like(p)
        if dtype == torch.bfloat16:
            tol = tol + BF * ref.abs()
        close(f.view, ref, tol, f"{act} {R}x{C}")
        assert f.intact()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,group", [("int8", 128), ("e4m3", 32), ("int8", 64)])
def test_act_bwd(act, dtype, fmt, group):
    for i, (R, C) in enumerate(SHAPES):
        dy = randn((R, C), 300 + i, dtype=dtype)
        ck, codes, scale = new_ckpt(R, C, fmt, group)
        aqfq.aqfq_ckpt8_pack(ck, _x(R, C, 400 + i).to(DEV))
        odd = i % 3 == 0
        fd = Framed(R, C, dtype, 5 if odd else 0, 3 if odd else 0, dy)
        fx = Framed(R, C, dtype, 1 if odd else 8, 0)
        fy = Framed(R, C, dtype)
        db = Framed(1, C, torch.float32)
        w = ws(aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(R, C))
        acc = i % 2 == 1
        db.view.fill_(0.75 if acc else float("nan"))
        aqfq.aqfq_ckpt8_act_bwd(ck, ACTS[act], fd.view, dx=fx.view, y=fy.view, dbias=db.view[0],
                                accumulate=acc, workspace=w)
        torch.cuda.synchronize()
        p = kept(codes, scale, fmt, group)
        d, ref = dact64(p, act), dy.double() * dact64(p, act)
        derr = 0.0 if act in ("none", "relu") else ACT_ERR
        e = dy.double().abs() * (derr + 4 * U * d.abs())
        close(fx.view, ref, e + (BF * ref.abs() if dtype == torch.bfloat16 else 0), f"dx {R}x{C}")
        y = act64(p, act)
        close(fy.view, y, p.abs() * derr + (BF * y.abs() if dtype == torch.bfloat16 else 0), "y")
        close(db.view[0], ref.sum(0) + (0.75 if acc else 0),
              e.sum(0) + (R + 64) * U * (ref.abs().sum(0) + 0.75), "dbias")
        assert fx.intact() and fy.intact() and db.intact()


def test_act_bwd_parts_alone():
    """Each output alone is what it is together; no checkpoint: plain column sums."""
    R, C = 300, 520
    dy = randn((R, C), 1).to(DEV)
    ck, codes, scale = new_ckpt(R, C, "int8", 32)
    aqfq.aqfq_ckpt8_pack(ck, _x(R, C, 2).to(DEV))
    w = ws(aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(R, C))
    a = [torch.empty(R, C, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    b = [torch.empty(C, device=DEV) for _ in range(3)]
    g = aqfq.ACT_SILU
    aqfq.aqfq_ckpt8_act_bwd(ck, g, dy, dx=a[0], y=a[1], dbias=b[0], workspace=w)
    aqfq.aqfq_ckpt8_act_bwd(ck, g, dy, dx=a[2])
    aqfq.aqfq_ckpt8_act_bwd(ck, g, dy, y=a[3])
    aqfq.aqfq_ckpt8_act_bwd(ck, g, dy, dbias=b[1], workspace=w)
    aqfq.aqfq_ckpt8_act_bwd(None, aqfq.ACT_NONE, dy, dbias=b[2], workspace=w)
    torch.cuda.synchronize()
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3]) and torch.equal(b[0], b[1])
    ref = dy.double().sum(0)
    close(b[2], ref, (R + 64) * U * dy.double().abs().sum(0))


def test_gradient_against_differences():
    """act' from the kernel against central differences of the 64-bit activation
    at the kept values: their error is h^2 |act'''| / 6 + 2^-53 |act| / h."""
    R, C = 8, 256
    ck, codes, scale = new_ckpt(R, C, "int8", 128)
    aqfq.aqfq_ckpt8_pack(ck, (randn((R, C), 5, 2.0, torch.float32)).to(DEV))
    p, h = kept(codes, scale, "int8", 128), 1e-5
    one, dx = torch.ones(R, C, device=DEV), torch.empty(R, C, device=DEV)
    for act in ("gelu", "gelu_tanh", "silu"):
        aqfq.aqfq_ckpt8_act_bwd(ck, ACTS[act], one, dx=dx)
        diff = (act64(p + h, act) - act64(p - h, act)) / (2 * h)
        close(dx, diff, torch.full_like(p, ACT_ERR + 1e-9 + 1e-9), act)


def test_empty_and_zero_rows():
    ck, codes, scale = new_ckpt(0, 40, "int8", 32)
    e = torch.empty(0, 40, device=DEV)
    aqfq.aqfq_ckpt8_pack(ck, e)
    aqfq.aqfq_ckpt8_unpack(ck, e)
    db = torch.full((40,), 3.0, device=DEV)
    w = ws(16)
    aqfq.aqfq_ckpt8_act_bwd(ck, aqfq.ACT_GELU, e, dx=e, dbias=db, accumulate=True, workspace=w)
    assert bool((db == 3).all())
    aqfq.aqfq_ckpt8_act_bwd(ck, aqfq.ACT_GELU, e, dx=e, dbias=db, workspace=w)
    assert bool((db == 0).all())
    ck, codes, scale = new_ckpt(4, 0, "int8", 32)
    z = torch.empty(4, 0, device=DEV)
    aqfq.aqfq_ckpt8_pack(ck, z)
    aqfq.aqfq_ckpt8_act_bwd(ck, aqfq.ACT_GELU, z, dx=z)
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits():
    """Two rows more than 2^32 elements apart."""
    C, ld = 72, (1 << 32) + 64
    big = torch.empty(ld + C, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((2, C), (ld, 1))
    src = randn((2, C), 9)
    x.copy_(src)
    ck, codes, scale = new_ckpt(2, C, "e4m3", 64)
    aqfq.aqfq_ckpt8_pack(ck, x)
    q, s = pack_ref(src, "e4m3", 64)
    np.testing.assert_array_equal(grid_values(codes, "e4m3"), q)
    aqfq.aqfq_ckpt8_unpack(ck, x)
    torch.cuda.synchronize()
    assert torch.equal(x.cpu(), kept(codes, scale, "e4m3", 64).bfloat16())


def test_same_bits_again_and_on_another_stream():
    R, C = 3000, 1003
    dy, x = randn((R, C), 11).to(DEV), _x(R, C, 12, torch.bfloat16).to(DEV)
    out = []
    for st in (None, torch.cuda.Stream(), None):
        ck, codes, scale = new_ckpt(R, C, "int8", 64)
        dx, db = torch.empty_like(dy), torch.empty(C, device=DEV)
        w = ws(aqfq.aqfq_ckpt8_act_bwd_workspace_bytes(R, C))
        torch.cuda.synchronize()
        aqfq.aqfq_ckpt8_pack(ck, x, stream=st)
        aqfq.aqfq_ckpt8_act_bwd(ck, aqfq.ACT_GELU, dy, dx=dx, dbias=db, workspace=w, stream=st)
        torch.cuda.synchronize()
        out.append((codes, scale, dx, db))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], o))


@pytest.mark.parametrize("fmt", [aqfq.INT8, aqfq.FP8_E4M3])
def test_unpack_of_many_rows_equals_its_slices(fmt):
    # 17 million elements take 16 columns per lane, the slices 8: the same arithmetic
    R, C, group = 16401, 1040, 64
    x = torch.randn(R, C, device="cuda").bfloat16()
    codes = torch.empty(R, C, dtype=torch.uint8, device="cuda")
    scale = torch.empty(R, -(-C // group), device="cuda")
    ck = aqfq.ckpt8(fmt, group, codes, scale)
    aqfq.aqfq_ckpt8_pack(ck, x)
    for act in (aqfq.ACT_NONE, aqfq.ACT_SILU):
        whole = torch.full_like(x, float("nan"))
        parts = torch.full_like(x, float("nan"))
        aqfq.aqfq_ckpt8_unpack(ck, whole, act=act)
        for lo in range(0, R, 6000):
            hi = min(R, lo + 6000)
            aqfq.aqfq_ckpt8_unpack(aqfq.ckpt8(fmt, group, codes[lo:hi], scale[lo:hi]),
                                   parts[lo:hi], act=act)
        assert torch.equal(whole.view(torch.int16), parts.view(torch.int16))

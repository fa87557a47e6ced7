"""The smooth activations over their whole range, tails included, in every call that computes
them: relative bounds, where the other tests' are absolute.

BF16 outputs: the arithmetic before the rounding is at most E = 2^-15 of the value off (an
exponential's argument of up to 122 is rounded three times: 3 x 122 x 2^-24 ln 2 of the value;
polynomials and reciprocals 2^-17), so the output lies between the rounded ends of that
interval.  Below binary32's normal range factors are flushed to zero: 2^-126 of what the
formula multiplies them with, |p| for a value; for a derivative |p| z' too, where tanh gelu's
inner derivative z' grows to 38 at -13."""
import math

import pytest
import torch

from layerlib import ACTS, DEV, U, act64, close, kept, new_ckpt, ws
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu
SMOOTH = ["gelu", "gelu_tanh", "silu"]
E = 2.0 ** -15
LEAST = 2.0 ** -126


def between(got, ref, e, what=""):
    """The BF16 output is a rounding of some value within e of ref."""
    lo, hi = (ref - e).bfloat16().double(), (ref + e).bfloat16().double()
    got = got.double().cpu()
    out = ~((got >= lo) & (got <= hi))
    assert not bool(out.any()), (what, int(out.sum()), got[out][:4], ref[out][:4])


def terms(p, act):
    """Two 64-bit terms whose sum is the derivative, and what multiplies their smallest factors."""
    p = p.double()
    if act == "gelu":
        return (0.5 * torch.special.erfc(-p / math.sqrt(2.0)),
                p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi), 1 + p.abs())
    c = math.sqrt(2 / math.pi)
    z = p if act == "silu" else 2 * c * (p + 0.044715 * p ** 3)
    dz = torch.ones_like(p) if act == "silu" else 2 * c * (1 + 3 * 0.044715 * p * p)
    return torch.sigmoid(z), p * dz * torch.sigmoid(z) * torch.sigmoid(-z), 1 + p.abs() * (1 + dz)


def value64(p, act):
    """act64 without its cancellation: tanh gelu as p sigmoid(2 u)."""
    return p.double() * terms(p, act)[0] if act != "gelu" else act64(p, act)


def sweep(rows, cols, lo=-13.0, hi=13.0):
    """Values all over [lo, hi], each group of 32 with its own largest one."""
    g = torch.Generator().manual_seed(rows * cols)
    x = lo + (hi - lo) * torch.rand(rows, cols, generator=g)
    size = torch.linspace(0.05, 1.0, rows * cols // 32).repeat_interleave(32).view(rows, cols)
    return torch.where(torch.rand(rows, cols, generator=g) < 0.5, x, x * size)


def checkpoint(rows, cols, fmt="int8"):
    ck, codes, scale = new_ckpt(rows, cols, fmt, 32)
    aqfq.aqfq_ckpt8_pack(ck, sweep(rows, cols).to(DEV))
    torch.cuda.synchronize()
    return ck, kept(codes, scale, fmt, 32)


# one to 16 columns per lane
@pytest.mark.parametrize("rows,cols", [(40, 288), (33, 1003 // 32 * 32), (4100, 4096)])
@pytest.mark.parametrize("act", SMOOTH)
def test_recomputed_in_bf16(rows, cols, act):
    for pad in (0, 1):
        ck, p = checkpoint(rows, cols)
        y = torch.empty(rows, cols + pad, dtype=torch.bfloat16, device=DEV)[:, :cols]
        aqfq.aqfq_ckpt8_unpack(ck, y, act=ACTS[act])
        torch.cuda.synchronize()
        ref = value64(p, act)
        between(y, ref, E * ref.abs() + LEAST * (1 + p.abs()), act)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_many_elements_recomputed_exactly(act, fmt):
    """16 columns per lane (2^24 elements and more)."""
    ck, p = checkpoint(4100, 4096, fmt)
    y = torch.empty(4100, 4096, dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_ckpt8_unpack(ck, y, act=ACTS[act])
    torch.cuda.synchronize()
    assert torch.equal(y.cpu(), act64(p, act).bfloat16())


@pytest.mark.parametrize("rows,cols", [(40, 288), (600, 1024)])
@pytest.mark.parametrize("act", SMOOTH)
def test_gradient_in_bf16(rows, cols, act):
    ck, p = checkpoint(rows, cols)
    one = torch.ones(rows, cols, dtype=torch.bfloat16, device=DEV)
    dx, y = torch.empty_like(one), torch.empty_like(one)
    aqfq.aqfq_ckpt8_act_bwd(ck, ACTS[act], one, dx=dx, y=y)
    torch.cuda.synchronize()
    a, b, amp = terms(p, act)
    between(dx, a + b, E * (a.abs() + b.abs()) + LEAST * amp, "dx")
    ref = value64(p, act)
    between(y, ref, E * ref.abs() + LEAST * (1 + p.abs()), "y")


# the products' epilogues: x is zero, the bias (or the kept pre-activation and a product of
# ones) gives the argument; sizes for the small tiles, split and whole, and for pairs of CTAs
@pytest.mark.parametrize("M,N", [(3, 4096), (1000, 1536), (4096, 4096), (4095, 4104)])
@pytest.mark.parametrize("act", SMOOTH)
def test_forward_epilogue(M, N, act):
    bias = torch.linspace(-13, 13, N)
    x = torch.zeros(M, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(N, 64, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_linear_fwd(x, w, y, bias=bias.to(DEV), act=ACTS[act],
                         workspace=ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_FWD, M, N, 64)))
    torch.cuda.synchronize()
    ref = value64(bias, act)
    assert bool((y == y[0]).all())
    between(y[0], ref, E * ref.abs() + LEAST * (1 + bias.abs()), act)


@pytest.mark.parametrize("M,K", [(3, 4096), (1000, 1536), (4096, 4096), (4095, 4104)])
@pytest.mark.parametrize("act", SMOOTH)
def test_input_gradient_epilogue(M, K, act):
    rows = min(M, 64)
    ck, codes, scale = new_ckpt(M, K, "int8", 32)
    x = sweep(rows, K // 32 * 32)
    x = torch.cat([x, torch.zeros(rows, K - x.shape[1])], 1)
    aqfq.aqfq_ckpt8_pack(ck, x.repeat(-(-M // rows), 1)[:M].contiguous().to(DEV))
    torch.cuda.synchronize()
    p = kept(codes[:rows], scale[:rows], "int8", 32)
    dy = torch.zeros(M, 64, dtype=torch.bfloat16, device=DEV)
    dy[:, 0] = 1.0
    w = torch.ones(64, K, dtype=torch.bfloat16, device=DEV)
    dx = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_linear_dgrad(dy, w, dx, act=ACTS[act], ckpt=ck,
                           workspace=ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_DGRAD, M, 64, K)))
    torch.cuda.synchronize()
    a, b, amp = terms(p, act)
    between(dx[:rows], a + b, E * (a.abs() + b.abs()) + LEAST * amp, act)
    assert torch.equal(dx[rows:], dx[:M - rows] if M % rows == 0 else dx[:rows].repeat(-(-M // rows), 1)[rows:M])


# FP32 outputs, U the unit roundoff of binary32.  An exponential 2^z of a z that is r times
# rounded is (4 + r |z| ln 2) U of itself off (the hardware's 2^-22 is 4 U), its reciprocal 2 U.
#   gelu       |p| <= 1.5: Phi = 1/2 + p C, 3 U and the fit's 7e-10; beyond, the tail: the fit's
#              2.4e-7 (4 U), reciprocal and eight roundings (12 U), exponential (z = p^2 / 2 log2 e,
#              3 times rounded); its complement one rounding more
#   tanh gelu  z four times rounded; the gate and its complement (with 2^z) from it
#   silu       z twice rounded; 1 - s as it is
def bounds_f32(p, act):
    p = p.double()
    a, b, amp = terms(p, act)
    y, d = p * a, a + b
    if act == "gelu":
        tail = (16 + 1.5 * p * p) * torch.minimum(a, 1 - a)
        phi = torch.where(p.abs() <= 1.5, torch.full_like(p, 3 + 7e-10 / U), tail + (p > 0))
        ev, ed = p.abs() * phi + y.abs(), phi + (6 + 1.5 * p * p) * b.abs() + d.abs()
    elif act == "gelu_tanh":
        z = (2 * math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)).abs()
        ev, ed = (4 * z + 9) * y.abs(), (4 * z + 8) * a + (8 * z + 26) * b.abs() + d.abs()
    else:
        t, n = 1 - a, p.abs()
        inner = 1 + p * t
        ev = (2 * n + 9) * y.abs()
        ed = a * (n * (t * a * (2 * n + 4) + 3 * a + 1) + inner.abs() + n * t) + (2 * n + 9) * d.abs()
    return U * ev + LEAST * (1 + p.abs()), U * ed + LEAST * amp


@pytest.mark.parametrize("rows,cols", [(40, 288), (33, 992), (600, 1024)])
@pytest.mark.parametrize("act", SMOOTH)
def test_fp32_outputs(rows, cols, act):
    for pad in (0, 1):
        ck, p = checkpoint(rows, cols)
        new = lambda: torch.empty(rows, cols + pad, device=DEV)[:, :cols]
        one, y, y2, dx = new().fill_(1.0), new(), new(), new()
        aqfq.aqfq_ckpt8_unpack(ck, y, act=ACTS[act])
        aqfq.aqfq_ckpt8_act_bwd(ck, ACTS[act], one, dx=dx, y=y2)
        torch.cuda.synchronize()
        a, b, _ = terms(p, act)
        ev, ed = bounds_f32(p, act)
        close(y, value64(p, act), ev, "value")
        close(y2, value64(p, act), ev, "value")
        close(dx, a + b, ed, "derivative")


@pytest.mark.parametrize("act", SMOOTH)
def test_fp32_outputs_of_large_arguments(act):
    """Far beyond the range where the formulas change: p or 0, 1 or 0."""
    x = torch.zeros(4, 32)
    x[0, :2] = torch.tensor([3e38, -3e38])
    x[1, :2] = torch.tensor([1e20, -1e20])
    x[2, :2] = torch.tensor([200.0, -200.0])
    x[3, :2] = torch.tensor([20.0, -20.0])
    ck, codes, scale = new_ckpt(4, 32, "int8", 32)
    aqfq.aqfq_ckpt8_pack(ck, x.to(DEV))
    torch.cuda.synchronize()
    p = kept(codes, scale, "int8", 32)
    one, y, dx = torch.ones(4, 32, device=DEV), torch.empty(4, 32, device=DEV), torch.empty(4, 32, device=DEV)
    aqfq.aqfq_ckpt8_act_bwd(ck, ACTS[act], one, dx=dx, y=y)
    torch.cuda.synchronize()
    close(y[:, 0], p[:, 0], 2 * U * p[:, 0].abs())
    close(dx[:, 0], torch.ones(4), torch.full((4,), 1e-7))
    close(y[:, 1], torch.zeros(4), torch.full((4,), 1e-7))
    close(dx[:, 1], torch.zeros(4), torch.full((4,), 1e-7))

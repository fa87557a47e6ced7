"""Shared by the tests of the layer calls: 64-bit restatements of the formulas
(plain torch on the CPU), the 8-bit grids as tables, and strided test buffers
whose surroundings are checked after a call."""
import math

import numpy as np
import torch

from learnable_scale_fake_gb300 import aqfq

DEV = "cuda:0"
U = 2.0 ** -24       # unit roundoff of binary32
BF = 2.0 ** -8       # BF16 rounding (half an ulp is at most 2^-9 of the value)
ACTS = {"none": aqfq.ACT_NONE, "relu": aqfq.ACT_RELU, "gelu": aqfq.ACT_GELU,
        "gelu_tanh": aqfq.ACT_GELU_TANH, "silu": aqfq.ACT_SILU}
FMTS = {"int8": aqfq.INT8, "e4m3": aqfq.FP8_E4M3}
QMAX = {"int8": 127.0, "e4m3": 448.0}
# the activations' approximations: exponentials, reciprocals and the polynomial of the normal
# distribution function (below 1.5e-7) leave value / x and derivative within 2^-18
ACT_ERR = 2.0 ** -18


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen(seed)) * std).to(dtype)


class Framed:
    """A [rows, cols] view with a row stride and an offset inside a larger buffer that holds a
    sentinel everywhere else; intact() says whether only the view was written."""

    def __init__(self, rows, cols, dtype, pad=0, off=0, src=None):
        self.ld = cols + pad
        n = off + max(rows, 1) * self.ld + 64
        esize = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n * esize,), 0xA5, dtype=torch.uint8, device=DEV)
        self.whole = self.raw.view(dtype)
        self.view = self.whole.as_strided((rows, cols), (self.ld, 1), off)
        self.mask = torch.ones(n, dtype=torch.bool, device=DEV)
        self.mask.as_strided((rows, cols), (self.ld, 1), off).fill_(False)
        if src is not None:
            self.view.copy_(src)
        self.esize = esize

    def intact(self):
        b = self.raw.view(-1, self.esize)[self.mask]
        return bool((b == 0xA5).all())


def act64(p, act):
    p = p.double()
    if act == "relu":
        return torch.where(p < 0, torch.zeros_like(p), p)
    if act == "gelu":
        return p * 0.5 * torch.special.erfc(-p / math.sqrt(2.0))
    if act == "gelu_tanh":
        return 0.5 * p * (1 + torch.tanh(math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)))
    if act == "silu":
        return p * torch.sigmoid(p)
    return p


def dact64(p, act):
    p = p.double()
    if act == "relu":
        return (p > 0).double()
    if act == "gelu":
        return (0.5 * torch.special.erfc(-p / math.sqrt(2.0))
                + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (p + 0.044715 * p ** 3))
        return 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * c * (1 + 0.134145 * p * p)
    if act == "silu":
        s = torch.sigmoid(p)
        return s * (1 + p * (1 - s))
    return torch.ones_like(p)


def _e4m3_table():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append((-a if c & 128 else a) if (c & 127) != 127 else math.nan)
    return np.array(v)


E4M3 = _e4m3_table()


def grid_values(codes, fmt):
    c = codes.cpu().numpy()
    return c.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[c]


def round_to_grid(v, fmt):
    """Nearest grid value of float64 v, ties to the even code, saturating."""
    if fmt == "int8":
        return np.clip(np.rint(v), -127, 127)
    pos = E4M3[:127]
    a = np.minimum(np.abs(v), 448.0)
    i = np.clip(np.searchsorted(pos, a, side="right") - 1, 0, 125)
    lo, hi = pos[i], pos[i + 1]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    return np.copysign(np.where(up, hi, lo), v)


def pack_ref(x, fmt, group):
    """(grid values, scales) of a float32 array by the definition."""
    x = x.float().cpu().numpy()
    R, C = x.shape
    q, n = np.zeros((R, C)), -(-C // group)
    scale = np.zeros((R, n), np.float32)
    with np.errstate(all="ignore"):
        for g in range(n):
            t = x[:, g * group:(g + 1) * group]
            amax = np.abs(t).max(1)
            bad = ~np.isfinite(t).all(1)
            s = np.where(bad, np.float32(np.nan), amax / np.float32(QMAX[fmt])).astype(np.float32)
            scale[:, g] = s
            v = (t / s[:, None]).astype(np.float32).astype(np.float64)
            v = np.where((s > 0)[:, None], v, 0.0)
            q[:, g * group:(g + 1) * group] = round_to_grid(v, fmt)
    return q, scale


def kept(codes, scale, fmt, group):
    """The values a checkpoint stands for: code * scale rounded to binary32, as float64."""
    q = grid_values(codes, fmt).astype(np.float32)
    s = scale.cpu().numpy()
    col = np.arange(q.shape[1]) // group
    with np.errstate(all="ignore"):
        return torch.from_numpy((q * s[:, col]).astype(np.float32)).double()


def new_ckpt(rows, cols, fmt, group):
    codes = torch.full((rows, cols), 0x5A, dtype=torch.uint8, device=DEV)
    scale = torch.full((rows, -(-cols // group)), -7.0, device=DEV)
    return aqfq.ckpt8(FMTS[fmt], group, codes, scale), codes, scale


def ws(nbytes):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=DEV)


def close(got, ref, tol, what=""):
    """|got - ref| <= tol elementwise; NaN and infinities of ref have to be met."""
    got, ref, tol = got.double().cpu(), ref.double().cpu(), tol.double().cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = ~fin & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    if fin.any():
        over = ((got - ref).abs() - tol)[fin]
        assert bool((over <= 0).all()), (
            f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, worst by {over.max()}")

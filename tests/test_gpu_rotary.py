"""Rotary positions against complex numbers in 64 bits.

Bounds (U the unit roundoff of binary32).  The angle in half turns is rounded to binary32 (at
most U / 2 in [-1, 1], pi U / 2 in the angle) and cut after 32 bits of a turn (2 pi 2^-32); sine and
cosine are within 2 ulp (4 U at most), so each is off by less than 6 U.  They are multiplied by
mscale (U), by an element (U each) and added (U): the pair (a, b) gives a value off by
(6 + 3) U mscale (|a| + |b|).  The angle itself, pos freqs: freqs / 2 pi in binary64 and the fraction's
last bit, and the reference's own binary64 product and reduction, 2^-50 of the angle.  A BF16
value is rounded by half a step at the end: finfo(bfloat16).eps / 2 = 2^-8 of it (the elements
that pass through are exact)."""
import math

import pytest
import torch

from layerlib import BF, DEV, U, close, gen
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu
LAYOUTS = {"half": aqfq.ROTARY_HALF, "interleaved": aqfq.ROTARY_INTERLEAVED}
# T, heads of q, heads of k (0: none), D, rot
SHAPES = [(1, 32, 8, 128, 128), (7, 3, 1, 64, 64), (33, 5, 0, 80, 42), (5, 2, 2, 81, 40), (300, 9, 3, 96, 48),
          (1, 1, 0, 2, 2), (4, 1, 1, 1, 0), (17, 40, 8, 16, 8), (3, 2, 1, 256, 256), (2, 3, 0, 7, 4),
          (2000, 6, 2, 64, 32), (2, 1, 1, 4096, 4094), (3, 0, 2, 32, 32), (0, 4, 2, 32, 32),
          # two elements at a time by halves in BF16
          (9, 5, 2, 128, 44), (300, 3, 1, 80, 36), (2, 17, 0, 12, 4), (5, 2, 2, 96, 92)]


def rotated(x, pos, freqs, layout, mscale, transposed):
    """(value, bound) in 64 bits of heads x [T, H, D]."""
    x, rot = x.double(), 2 * len(freqs)
    angle = pos.double()[:, None] * freqs
    turn = torch.polar(torch.full_like(angle, mscale), -angle if transposed else angle)[:, None]
    z, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = z[..., :rot // 2], z[..., rot // 2:]
    else:
        a, b = z[..., 0::2], z[..., 1::2]
    w = torch.complex(a.contiguous(), b.contiguous()) * turn
    size = abs(mscale) * (a.abs() + b.abs())
    err = size * (9 * U + 2.0 ** -50 * angle.abs()[:, None])

    def laid(p, q):
        return torch.cat([p, q], -1) if layout == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([laid(w.real, w.imag), rest], -1), torch.cat([laid(err, err), 0 * rest], -1)


def heads(T, H, D, dtype, seed):
    return (torch.randn((T, H, D), generator=gen(seed)) * 2).to(dtype)


class Placed:
    """[T, H, D] inside a larger buffer of a sentinel: token-major or head-major, with gaps."""

    def __init__(self, T, H, D, dtype, form, src=None):
        off, gap, head_major = form
        hs = D + gap
        ld = H * hs + 2 * gap
        if head_major:
            ld, hs = D + gap, T * (D + gap) + gap
        n = off + max(T, 1) * ld + max(H, 1) * hs + 64
        self.whole = torch.full((n,), -77.0, dtype=dtype, device=DEV)
        self.view = self.whole.as_strided((T, H, D), (ld, hs, 1), off)
        self.mask = torch.ones(n, dtype=torch.bool, device=DEV)
        self.mask.as_strided((T, H, D), (ld, hs, 1), off).fill_(False)
        if src is not None:
            self.view.copy_(src)

    def intact(self):
        return bool((self.whole[self.mask] == -77.0).all())


# offset, gap, head-major: aligned to 16 bytes, to 8 (BF16), odd; a [heads, T, D] tensor
FORMS = [(0, 0, False), (8, 8, False), (4, 4, False), (1, 3, False), (0, 0, True), (2, 1, True)]


def positions(T, far, seed):
    if far:
        return torch.randint(-(1 << 31), 1 << 31, (T,), generator=gen(seed))
    return torch.arange(T) * 3 + 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("form", FORMS)
def test_against_complex_numbers(dtype, layout, form):
    for i, (T, Hq, Hk, D, rot) in enumerate(SHAPES):
        transposed, mscale = i % 2 == 1, (1.0, 1.25, 0.0)[i % 3]
        freqs, _ = aqfq.aqfq_rotary_freqs(rot)
        pos = positions(T, i % 4 == 2, i)
        out, ref = [], []
        for H, seed in ((Hq, 50 + i), (Hk, 90 + i)):
            x = heads(T, H, D, dtype, seed)
            out.append((Placed(T, H, D, dtype, form, x), Placed(T, H, D, dtype, form)))
            ref.append((x, rotated(x, pos, freqs, layout, mscale, transposed)))
        kw = {} if Hk == 0 else {"k": out[1][0].view, "yk": out[1][1].view}
        aqfq.aqfq_rotary(out[0][0].view, pos.to(DEV), freqs.to(DEV), out[0][1].view, layout=LAYOUTS[layout],
                         mscale=mscale, transposed=transposed, **kw)
        torch.cuda.synchronize()
        for (fx, fy), (x, (want, tol)) in zip(out, ref):
            if fy.view.shape[1] == 0:
                continue
            if dtype == torch.bfloat16:
                tol = tol + BF * want.abs() * (tol > 0)
            close(fy.view, want, tol, f"{T} {H} {D} {rot}")
            assert fy.intact() and torch.equal(fx.view.cpu(), x)


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_gives_the_same_bits(dtype, layout):
    """Heads of one packed tensor, rotated where they are; the values and the rest stay."""
    for D, rot in ((64, 64), (80, 32), (33, 6)):
        T, Hq, Hk = 19, 6, 2
        qkv = heads(T, Hq + 2 * Hk, D, dtype, 7).to(DEV)
        before = qkv.clone()
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        pos, freqs = torch.arange(T, device=DEV), aqfq.aqfq_rotary_freqs(rot)[0].to(DEV)
        yq, yk = torch.empty_like(q), torch.empty_like(k)
        aqfq.aqfq_rotary(q, pos, freqs, yq, k=k, yk=yk, layout=LAYOUTS[layout])
        aqfq.aqfq_rotary(q, pos, freqs, q, k=k, yk=k, layout=LAYOUTS[layout])
        torch.cuda.synchronize()
        assert torch.equal(q, yq) and torch.equal(k, yk)
        assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_transposed_is_the_gradient():
    """<dy, R x> = <R^T dy, x>, and differences of the call itself."""
    T, H, D, rot = 40, 4, 48, 30
    freqs, pos = aqfq.aqfq_rotary_freqs(rot)[0].to(DEV), torch.randint(0, 1 << 20, (T,), generator=gen(3)).to(DEV)
    for layout in LAYOUTS.values():
        x, d, dy = (heads(T, H, D, torch.float32, s).to(DEV) for s in (1, 2, 3))
        out = []
        for t, tr in ((x, False), (x + d, False), (dy, True)):
            y = torch.empty_like(t)
            aqfq.aqfq_rotary(t, pos, freqs, y, layout=layout, mscale=1.5, transposed=tr)
            out.append(y.double())
        torch.cuda.synchronize()
        # both sides are sums of T H D terms of about 6, each off by about 2^-20 of itself
        n = T * H * D
        lhs, rhs = ((out[1] - out[0]) * dy.double()).sum(), (out[2] * d.double()).sum()
        assert abs(float(lhs - rhs)) <= 2.0 ** -20 * n * 8


def test_broadcast_heads_and_positions_far_away():
    """Heads read from one (stride 0), positions at the ends of 64 bits: the angle is a product
    modulo one turn, so a frequency of a quarter turn per position is exact."""
    T, H, D = 4, 3, 2
    x = heads(T, 1, D, torch.float32, 5).to(DEV)
    pos = torch.tensor([1, -3, (1 << 62) + 2, -(1 << 63)], device=DEV)
    freqs = torch.tensor([math.pi / 2], dtype=torch.float64, device=DEV)
    y = torch.empty(T, H, D, device=DEV)
    aqfq.aqfq_rotary(x.expand(T, H, D), pos, freqs, y)
    torch.cuda.synchronize()
    a, b = x.double()[:, 0, 0], x.double()[:, 0, 1]
    # a quarter, a quarter (-3), a half and no turn; 2^62 positions leave F's last bit 2^-2 turns off
    for t, (c, s) in enumerate(((0, 1), (0, 1))):
        want = torch.stack([a[t] * c - b[t] * s, a[t] * s + b[t] * c])
        assert float((y[t].double() - want).abs().max()) <= 2.0 ** -20
    assert bool(torch.isfinite(y).all())
    n = y.double().square().sum(-1)
    assert float((n / (a * a + b * b)[:, None] - 1).abs().max()) <= 2.0 ** -19


def test_non_finite_values_stay_in_their_pair():
    x = heads(3, 2, 64, torch.float32, 8)
    x[1, 0, 5], x[2, 1, 40] = float("nan"), float("inf")
    freqs = aqfq.aqfq_rotary_freqs(64)[0]
    y = torch.empty(3, 2, 64, device=DEV)
    aqfq.aqfq_rotary(x.to(DEV), torch.tensor([3, 4, 5], device=DEV), freqs.to(DEV), y)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y.cpu())
    assert bad.nonzero().tolist() == [[1, 0, 5], [1, 0, 37], [2, 1, 8], [2, 1, 40]]


def test_captured_on_another_stream_and_replayed():
    T, Hq, Hk, D = 65, 8, 2, 128
    q, k = heads(T, Hq, D, torch.bfloat16, 1).to(DEV), heads(T, Hk, D, torch.bfloat16, 2).to(DEV)
    pos, freqs = torch.arange(T, device=DEV), aqfq.aqfq_rotary_freqs(D)[0].to(DEV)
    yq, yk, zq, zk = (torch.empty_like(t) for t in (q, k, q, k))
    aqfq.aqfq_rotary(q, pos, freqs, zq, k=k, yk=zk)
    g = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        aqfq.aqfq_rotary(q, pos, freqs, yq, k=k, yk=yk)
    for shift in (0, 11):
        pos.copy_(torch.arange(T) + shift)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        aqfq.aqfq_rotary(q, pos, freqs, zq, k=k, yk=zk)
        torch.cuda.synchronize()
        assert torch.equal(yq, zq) and torch.equal(yk, zk)


def test_offsets_beyond_32_bits():
    """Tokens 2^25 elements apart: the last starts beyond 2^32 bytes and 2^31 elements."""
    T, D, ld = 70, 64, 1 << 25
    whole = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV)
    x = whole.as_strided((T, 2, D), (ld, D, 1))
    x.copy_(heads(T, 2, D, torch.bfloat16, 4))
    pos, freqs = torch.arange(T, device=DEV) + 9, aqfq.aqfq_rotary_freqs(D)[0].to(DEV)
    packed, y, z = x.contiguous(), whole.as_strided((T, 2, D), (ld, D, 1), 4096), torch.empty(T, 2, D, dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_rotary(x, pos, freqs, y)
    aqfq.aqfq_rotary(packed, pos, freqs, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)

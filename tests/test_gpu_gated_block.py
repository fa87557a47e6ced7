"""The calls between a layer's quantized products together: the gated block in scale-only
training, and query and key heads from a norm through their rotation to the per-head quantizer
and back.

The reference repeats each in 64 bits from the same fake-quantized weights and, in the backward
pass, from what was kept.  Along any path at most eight tensors are rounded to BF16 (by at
most 2^-8 of a value, 2^-9 of its 2-norm on average); sums of them may cancel to about half their
size, so results agree to 16 * 2^-9 of their 2-norm."""
import pytest
import torch

from layerlib import act64, close, dact64, kept, randn, ws
from learnable_scale_fake_gb300 import aqfq, gated_block

pytestmark = pytest.mark.gpu
TOL = 16 * 2.0 ** -9


def rel(got, ref):
    ref = ref.double().cpu()
    return float((got.double().cpu() - ref).norm() / ref.norm())


def rms(t, eps):
    return 1 / torch.sqrt((t * t).mean(1, keepdim=True) + eps)


def rms_grad(t, r, d):
    """Gradient through t r of d."""
    n = t * r
    return r * (d - n * (d * n).mean(1, keepdim=True))


@pytest.mark.parametrize("tokens,hidden,ff,fmt,group", [(200, 256, 512, "int8", 128), (77, 128, 336, "e4m3", 64)])
def test_block_against_64_bits(tokens, hidden, ff, fmt, group):
    f = {"int8": aqfq.INT8, "e4m3": aqfq.FP8_E4M3}[fmt]
    b = gated_block.random_block(hidden, ff, tokens, seed=3, fmt=f, group=group, alpha=0.5)
    h, dh, dn = (randn((tokens, hidden), s).cuda() for s in (1, 2, 3))
    n = b.norm_in(h, torch.empty_like(h))
    h1, n1 = (t.clone() for t in b.forward(h, n))
    gh, gn = (t.clone() for t in b.backward(h, dh, dn))
    torch.cuda.synchronize()
    assert int(b.error.item()) == 0
    d = lambda t: t.double().cpu()
    w1, w2, eps = d(b.w1_hat), d(b.w2_hat), b.eps
    n0 = d(h) * rms(d(h), eps) * d(b.gamma_in)
    assert rel(n, n0) <= TOL
    p = n0 @ w1.T
    y = act64(p[:, :ff], "silu") * p[:, ff:]
    f0 = y @ w2.T
    assert rel(b.f, f0) <= TOL
    c = 0.5 * d(b.gate) * d(b.gamma_post)
    ref = d(h) + c * (f0 * rms(f0, eps))
    assert rel(h1, ref) <= TOL
    assert rel(n1, ref * rms(ref, eps) * d(b.gamma_pre)) <= TOL
    # backward, from what was kept
    hk, fk = d(h1), d(b.f)
    rh, rf = d(b.rstd_pre)[:, None], d(b.rstd_post)[:, None]
    dx = rms_grad(hk, rh, d(dn) * d(b.gamma_pre)) + d(dh)
    assert rel(gh, dx) <= TOL
    share = (dx * fk * rf).sum(0)
    for got, want in ((b.dgate, 0.5 * d(b.gamma_post) * share), (b.dgamma_post, 0.5 * d(b.gate) * share),
                      (b.dgamma_pre, (d(dn) * hk * rh).sum(0))):
        assert rel(got, want) <= TOL
    df = rms_grad(fk, rf, c * dx)
    assert rel(b.df, df) <= TOL
    kg, ku = (kept(*k.tensors, fmt, group) for k in (b.kept_gate, b.kept_up))
    hidden_act = act64(kg, "silu") * ku
    assert rel(b.dw2, df.T @ hidden_act) <= TOL
    s = df @ w2
    dp = torch.cat([s * ku * dact64(kg, "silu"), s * act64(kg, "silu")], 1)
    assert rel(b.dp, dp) <= TOL
    assert rel(b.dw1, dp.T @ n0) <= TOL
    assert rel(gn, dp @ w1) <= TOL
    # the scale gradients are those of the weights' gradients, bit for bit
    for w, dw, sc, g, ds in ((b.w1, b.dw1, b.s1, b.g1, b.ds1), (b.w2, b.dw2, b.s2, b.g2, b.ds2)):
        again = torch.empty_like(ds)
        aqfq.aqfq_scale_grad(gated_block.SPEC, w, dw, sc, g, dscale=again)
        assert torch.equal(again, ds)


def test_example_runs(capsys):
    gated_block.main(steps=3, hidden=256, ff=512, tokens=256)
    lines = [line for line in capsys.readouterr().out.splitlines() if "loss" in line]
    assert lines and all(float(line.split()[-1]) >= 0 for line in lines)


def test_block_on_another_stream_and_in_a_graph_gives_the_same_bits():
    b = gated_block.random_block(256, 512, 130, seed=4)
    h, dh, dn = (randn((130, 256), s).cuda() for s in (1, 2, 3))
    n = b.norm_in(h, torch.empty_like(h))

    def run(stream=None):
        b.forward(h, n, stream=stream)
        b.backward(h, dh, dn, stream=stream)

    outs = lambda: [t.clone() for t in (b.h_out, b.n_out, b.dh, b.dn, b.ds1, b.ds2, b.dgate, b.dgamma_pre)]
    run()
    torch.cuda.synchronize()
    first = outs()
    st = torch.cuda.Stream()
    run(st)
    torch.cuda.synchronize()
    second = outs()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for t in (b.h_out, b.n_out, b.dh, b.dn, b.ds1, b.ds2):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    third = outs()
    for a, c, e in zip(first, second, third):
        assert torch.equal(a, c) and torch.equal(a, e)


def test_heads_from_the_norm_to_the_per_head_quantizer_and_back():
    """norm -> query and key projection -> rotation in place -> per-head E4M3 fake-quant with learned
    scales; back: the straight-through gradient, the transposed rotation, the projection's gradients."""
    T, hidden, Hq, Hk, D = 96, 256, 6, 2, 64
    H = Hq + Hk
    h = randn((T, hidden), 1).cuda()
    gamma = (1 + randn((hidden,), 2, 0.1)).cuda()
    w = randn((H * D, hidden), 3, hidden ** -0.5).cuda()
    n, qk = torch.empty_like(h), torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
    pos = (torch.arange(T, device="cuda") * 7 + 100000)
    freqs, m = aqfq.aqfq_rotary_freqs(D, scaling=aqfq.ROTARY_PARTS, factor=4.0, length=8192.0)
    freqs = freqs.cuda()
    aqfq.aqfq_block_norm_fwd(h, None, 1e-6, y=n, gamma_pre=gamma)
    aqfq.aqfq_linear_fwd(n, w, qk, workspace=ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_FWD, T, H * D, hidden)))
    plain = qk.clone()
    heads = qk.view(T, H, D)
    aqfq.aqfq_rotary(heads[:, :Hq], pos, freqs, heads[:, :Hq], k=heads[:, Hq:], yk=heads[:, Hq:], mscale=m)
    lo, hi, scale = (torch.empty(H, device="cuda") for _ in range(3))
    aqfq.aqfq_observer_minmax(heads, lo, hi)
    aqfq.aqfq_minmax_scale(lo, hi, 448.0, scale)
    spec = aqfq.qspec(aqfq.FP8_E4M3, aqfq.PER_HEAD)
    hat = torch.empty_like(heads)
    aqfq.aqfq_qdq_fwd(spec, heads, scale, None, hat)
    torch.cuda.synchronize()
    # the heads, then what the quantizer sees
    d = lambda t: t.double().cpu()
    assert rel(plain, (d(h) * rms(d(h), 1e-6) * d(gamma)) @ d(w).T) <= TOL
    turn = torch.polar(torch.full((T, D // 2), m, dtype=torch.float64), torch.outer(d(pos), d(freqs)))[:, None]
    z = d(plain).view(T, H, D)
    r = torch.complex(z[..., :D // 2].contiguous(), z[..., D // 2:].contiguous()) * turn
    turned = torch.cat([r.real, r.imag], -1)
    close(heads, turned, 2.0 ** -8 * turned.abs() + 2.0 ** -20 * (z.abs() + z.roll(D // 2, -1).abs()) * m)
    assert torch.equal(hi.cpu(), heads.float().amax((0, 2)).cpu())
    # E4M3 holds each value to 2^-4 of itself, or half its smallest step
    close(hat, d(heads), (2.0 ** -4 + 2.0 ** -8) * d(heads).abs() + d(scale)[None, :, None] * 2.0 ** -10)
    # back
    dhat = randn((T, H, D), 9).cuda()
    ds, dx = torch.empty(H, device="cuda"), torch.empty_like(heads)
    aqfq.aqfq_scale_grad(spec, heads, dhat, scale, None, dscale=ds, dx=dx,
                         workspace=ws(aqfq.aqfq_scale_grad_workspace_bytes(spec, T, H, D)))
    back = dx.clone()
    aqfq.aqfq_rotary(dx[:, :Hq], pos, freqs, dx[:, :Hq], k=dx[:, Hq:], yk=dx[:, Hq:], mscale=m, transposed=True)
    dn, dw = torch.empty_like(n), torch.empty_like(w)
    flat = dx.view(T, H * D)
    aqfq.aqfq_linear_dgrad(flat, w, dn, workspace=ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_DGRAD, T, H * D, hidden)))
    aqfq.aqfq_linear_wgrad(flat, n, dw, workspace=ws(aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_WGRAD, T, H * D, hidden)))
    torch.cuda.synchronize()
    z = d(back)
    r = torch.complex(z[..., :D // 2].contiguous(), z[..., D // 2:].contiguous()) * turn.conj()
    g = torch.cat([r.real, r.imag], -1)
    assert rel(dx, g) <= TOL
    assert rel(dn, g.reshape(T, -1) @ d(w)) <= TOL
    assert rel(dw, g.reshape(T, -1).T @ d(n)) <= TOL

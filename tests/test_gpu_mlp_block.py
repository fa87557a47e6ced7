"""The layer calls together: a pre-norm MLP block in scale-only training.

The reference repeats the block in 64 bits from the same fake-quantized weights
and, in the backward pass, from the values that the 8-bit checkpoints hold.  Along
any path at most six tensors are rounded to BF16 (relative error at most 2^-9
each); sums of them may cancel to about half their size, so results agree to
12 * 2^-9 of their 2-norm."""
import pytest
import torch

from layerlib import act64, dact64, kept
from learnable_scale_fake_gb300 import aqfq, mlp_block

pytestmark = pytest.mark.gpu
TOL = 12 * 2.0 ** -9


def rel(got, ref):
    ref = ref.double().cpu()
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("tokens,hidden,ff,fmt,group", [(200, 256, 512, "int8", 128),
                                                        (77, 128, 336, "e4m3", 64)])
def test_block_against_64_bits(tokens, hidden, ff, fmt, group):
    f = {"int8": aqfq.INT8, "e4m3": aqfq.FP8_E4M3}[fmt]
    b = mlp_block.random_block(hidden, ff, tokens, seed=3, fmt=f, group=group)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    dy = torch.randn(tokens, hidden, device="cuda").bfloat16()
    y = b.forward(x).clone()
    dx = b.backward(dy).clone()
    torch.cuda.synchronize()
    assert int(b.error.item()) == 0
    d = lambda t: t.double().cpu()
    w1, w2, ga, be = d(b.w1_hat), d(b.w2_hat), d(b.gamma), d(b.beta)

    def norm(v):
        mu = v.mean(1, keepdim=True)
        r = 1 / torch.sqrt(((v - mu) ** 2).mean(1, keepdim=True) + b.eps)
        return mu, r, (v - mu) * r * ga + be

    mu, r, n = norm(d(x))
    pre = n @ w1.T + d(b.b1)
    assert rel(y, d(x) + act64(pre, "gelu") @ w2.T + d(b.b2)) <= TOL
    # backward, from what was kept
    kx = kept(*b.kept_x.tensors, fmt, group)
    kp = kept(*b.kept_pre.tensors, fmt, group)
    dpre = (d(dy) @ w2) * dact64(kp, "gelu")
    assert rel(b.dw2, d(dy).T @ act64(kp, "gelu")) <= TOL
    assert rel(b.dpre, dpre) <= TOL
    assert rel(b.dw1, dpre.T @ norm(kx)[2]) <= TOL
    u, h = (dpre @ w1) * ga, (kx - mu) * r
    ref = r * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True)) + d(dy)
    assert rel(dx, ref) <= TOL
    # the scale gradients are those of the weights' gradients, bit for bit
    ds = torch.empty_like(b.ds1)
    aqfq.aqfq_scale_grad(mlp_block.SPEC, b.w1, b.dw1, b.s1, b.g1, dscale=ds)
    assert torch.equal(ds, b.ds1)


def test_training_the_scales_lowers_the_loss(capsys):
    mlp_block.main(steps=11, hidden=256, ff=1024, tokens=512)
    loss = [float(line.split()[-1]) for line in capsys.readouterr().out.splitlines() if "loss" in line]
    assert loss[-1] < loss[0]


def test_block_on_another_stream_gives_the_same_bits():
    b = mlp_block.random_block(256, 512, 130, seed=4)
    x, dy = (torch.randn(130, 256, device="cuda").bfloat16() for _ in range(2))
    out = []
    for st in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        y = b.forward(x, stream=st)
        dx = b.backward(dy, stream=st)
        torch.cuda.synchronize()
        out.append([t.clone() for t in (y, dx, b.ds1, b.ds2)])
    assert all(torch.equal(p, q) for p, q in zip(*out))

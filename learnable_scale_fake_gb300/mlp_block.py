"""A pre-norm MLP block in scale-only training, run through the C ABI:

    y = x + act(norm(x) W1_hat^T + b1) W2_hat^T + b2

W1_hat and W2_hat are the NVFP4 fake-quant of frozen BF16 weights; only their
block scales train.  Between the forward and the backward pass the block keeps
x and the hidden pre-activation in 8 bits (one byte per element and one float
per `group` of them, 128 by default) and two floats per token; the norm's
output and the hidden activation are recomputed.

The backward pass sees x as its checkpoint gives it back, x~, in two places, and
not in the same way: the norm's output, an operand of the first weight's
gradient, is recomputed from x~ with the mean and deviation of x~; the norm's
own gradient forms h = (x~ - mean) rstd with those of the exact x, which the
forward kept.

``python -m learnable_scale_fake_gb300.mlp_block`` trains the scales of a small
block against its unquantized self and prints the loss.
(AngelSlim mcore_qad article, sections 1 and 2.3: frozen weights, fake-quant in
the forward, the gradient flows to the scales.)
"""
from __future__ import annotations

import torch

from . import aqfq

SPEC = aqfq.qspec(aqfq.NVFP4, aqfq.PER_GROUP, group=16)


class MlpBlock:
    """tokens x hidden activations, hidden -> ff -> hidden; every buffer is made once.

    ``fmt`` / ``group``: the 8-bit checkpoints' format (aqfq.INT8 or
    aqfq.FP8_E4M3) and group of columns.  hidden and ff are multiples of 16."""

    def __init__(self, w1, w2, gamma, beta, b1, b2, tokens, act=aqfq.ACT_GELU, fmt=aqfq.INT8,
                 group=128, eps=1e-5):
        self.w1, self.w2 = w1, w2
        self.gamma, self.beta, self.b1, self.b2 = gamma, beta, b1, b2
        self.act, self.eps = act, eps
        ff, hidden = w1.shape
        dev = w1.device

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=dev)

        def kept(cols):
            return aqfq.ckpt8(fmt, group, new(tokens, cols, dtype=torch.uint8),
                              new(tokens, -(-cols // group), dtype=torch.float32))

        # learned block scales and tensor scales, initialised from the weights
        self.s1, self.s2 = (new(w.numel() // 16, dtype=torch.float32) for w in (w1, w2))
        self.g1, self.g2 = new(1, dtype=torch.float32), new(1, dtype=torch.float32)
        aqfq.aqfq_scale_init(SPEC, w1, self.s1, self.g1)
        aqfq.aqfq_scale_init(SPEC, w2, self.s2, self.g2)
        self.ds1, self.ds2 = torch.empty_like(self.s1), torch.empty_like(self.s2)
        self.w1_hat, self.w2_hat = torch.empty_like(w1), torch.empty_like(w2)
        self.dw1, self.dw2 = torch.empty_like(w1), torch.empty_like(w2)
        # what lives from the forward to the backward pass
        self.kept_x, self.kept_pre = kept(hidden), kept(ff)
        self.mean, self.rstd = new(tokens, dtype=torch.float32), new(tokens, dtype=torch.float32)
        # scratch within a pass
        self.n, self.h = new(tokens, hidden), new(tokens, ff)
        self.dpre, self.dn = new(tokens, ff), new(tokens, hidden)
        self.y, self.dx = new(tokens, hidden), new(tokens, hidden)
        M = tokens
        need = max(aqfq.aqfq_linear_workspace_bytes(k, M, n, c)
                   for k in (aqfq.LINEAR_FWD, aqfq.LINEAR_DGRAD, aqfq.LINEAR_WGRAD)
                   for n, c in ((ff, hidden), (hidden, ff)))
        self.workspace = new(max(need, 16), dtype=torch.uint8)
        self.error = torch.zeros(1, dtype=torch.int32, device=dev)

    def kept_bytes(self) -> int:
        """Bytes held between the passes."""
        return sum(t.nbytes for c in (self.kept_x, self.kept_pre) for t in c.tensors) + \
            self.mean.nbytes + self.rstd.nbytes

    def forward(self, x, stream=None):
        kw = {"workspace": self.workspace, "error_flag": self.error, "stream": stream}
        aqfq.aqfq_qdq_fwd(SPEC, self.w1, self.s1, self.g1, self.w1_hat, stream=stream)
        aqfq.aqfq_qdq_fwd(SPEC, self.w2, self.s2, self.g2, self.w2_hat, stream=stream)
        aqfq.aqfq_layernorm_fwd(x, self.gamma, self.beta, self.eps, self.n, mean=self.mean,
                                rstd=self.rstd, ckpt=self.kept_x, stream=stream)
        aqfq.aqfq_linear_fwd(self.n, self.w1_hat, self.h, bias=self.b1, act=self.act,
                             ckpt=self.kept_pre, **kw)
        aqfq.aqfq_linear_fwd(self.h, self.w2_hat, self.y, bias=self.b2, residual=x, **kw)
        return self.y

    def backward(self, dy, stream=None):
        """dx, with the scale gradients in ds1 and ds2."""
        kw = {"workspace": self.workspace, "error_flag": self.error, "stream": stream}
        # hidden activation recomputed; the second weight's gradient and its scales'
        aqfq.aqfq_ckpt8_unpack(self.kept_pre, self.h, act=self.act, stream=stream)
        aqfq.aqfq_linear_wgrad(dy, self.h, self.dw2, **kw)
        aqfq.aqfq_scale_grad(SPEC, self.w2, self.dw2, self.s2, self.g2, dscale=self.ds2, stream=stream)
        # through the second product and the activation in one call
        aqfq.aqfq_linear_dgrad(dy, self.w2_hat, self.dpre, act=self.act, ckpt=self.kept_pre, **kw)
        # norm's output recomputed; the first weight
        aqfq.aqfq_ckpt8_unpack(self.kept_x, self.dn, stream=stream)
        aqfq.aqfq_layernorm_fwd(self.dn, self.gamma, self.beta, self.eps, self.n, stream=stream)
        aqfq.aqfq_linear_wgrad(self.dpre, self.n, self.dw1, **kw)
        aqfq.aqfq_scale_grad(SPEC, self.w1, self.dw1, self.s1, self.g1, dscale=self.ds1, stream=stream)
        # through the first product and the norm; the residual branch joins in
        aqfq.aqfq_linear_dgrad(self.dpre, self.w1_hat, self.dn, **kw)
        aqfq.aqfq_layernorm_bwd(self.dn, None, self.mean, self.rstd, self.gamma, self.dx, dres=dy,
                                ckpt=self.kept_x, stream=stream)
        return self.dx


def random_block(hidden, ff, tokens, seed=0, dev="cuda", **kw):
    g = torch.Generator(device=dev).manual_seed(seed)

    def n(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).bfloat16()

    return MlpBlock(n(ff, hidden, std=hidden ** -0.5), n(hidden, ff, std=ff ** -0.5),
                    1 + n(hidden, std=0.1), n(hidden, std=0.1), n(ff, std=0.1), n(hidden, std=0.1),
                    tokens, **kw)


def main(steps=20, hidden=2048, ff=8192, tokens=4096, lr=3e-3):
    block = random_block(hidden, ff, tokens)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    # the target: the same block with its weights as they are
    h, target = torch.empty_like(block.h), torch.empty_like(block.y)
    aqfq.aqfq_layernorm_fwd(x, block.gamma, block.beta, block.eps, block.n)
    aqfq.aqfq_linear_fwd(block.n, block.w1, h, bias=block.b1, act=block.act, workspace=block.workspace)
    aqfq.aqfq_linear_fwd(h, block.w2, target, bias=block.b2, residual=x, workspace=block.workspace)
    print(f"kept between the passes: {block.kept_bytes() / 2**20:.1f} MiB "
          f"(in BF16 {(hidden + ff) * tokens * 2 / 2**20:.1f} MiB)")
    opt = torch.optim.Adam([block.s1, block.s2], lr=lr * float(block.s1.mean()))
    for i in range(steps):
        diff = block.forward(x).float() - target.float()
        loss = diff.square().mean()
        block.backward((diff * (2.0 / diff.numel())).bfloat16())
        block.s1.grad, block.s2.grad = block.ds1, block.ds2
        opt.step()
        if i % 5 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {loss.item():.6f}")
    assert int(block.error.item()) == 0, "a pipeline wait timed out"


if __name__ == "__main__":
    main()

"""The linear products where the kernel is chosen by the size, and operands as torch makes them.
Bounds as in test_gpu_linear.py."""
import pytest
import torch

from layerlib import DEV, randn
from learnable_scale_fake_gb300 import aqfq

pytestmark = pytest.mark.gpu


def test_an_empty_inner_axis_of_contiguous_tensors():
    """torch's [rows, 0] tensors have a row stride of one element."""
    z = lambda r, c: torch.empty(r, c, dtype=torch.bfloat16, device=DEV)
    b, res = randn((40,), 1), randn((3, 40), 2)
    y = torch.full((3, 40), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert z(3, 0).stride() == (1, 1)
    aqfq.aqfq_linear_fwd(z(3, 0), z(40, 0), y, bias=b.to(DEV), act=aqfq.ACT_RELU, residual=res.to(DEV))
    dx = torch.full((5, 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    aqfq.aqfq_linear_dgrad(z(5, 0), z(0, 24), dx)
    dw = torch.full((16, 24), float("nan"), device=DEV)
    aqfq.aqfq_linear_wgrad(z(0, 16), z(0, 24), dw)
    # outputs without elements
    aqfq.aqfq_linear_dgrad(z(5, 16), z(16, 0), z(5, 0))
    aqfq.aqfq_linear_wgrad(z(8, 16), z(8, 0), z(16, 0))
    torch.cuda.synchronize()
    p = torch.clamp(b.double().expand(3, 40), min=0)
    assert torch.equal(y.cpu(), (p + res.double()).bfloat16())
    assert bool((dx == 0).all()) and bool((dw == 0).all())

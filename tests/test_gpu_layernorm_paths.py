"""Layer norm where the kernel is chosen by the size: workspaces at every alignment that the
header allows, rows whose mean times 1 / deviation overflows.  Bounds as in test_gpu_layernorm.py."""
import pytest
import torch

from layerlib import DEV, kept, new_ckpt, randn
from learnable_scale_fake_gb300 import aqfq
from test_gpu_layernorm import _case, _check_bwd, _stats

pytestmark = pytest.mark.gpu


# rows in registers with one group of warps per block (sums straight to scratch), several
# groups, odd widths, and both kinds of the ring
@pytest.mark.parametrize("R,C", [(60, 1160), (200, 4096), (20, 8192), (400, 512), (90, 1003),
                                 (700, 8192), (1300, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["none", "int8"])
def test_backward_workspace_at_any_multiple_of_8_bytes(R, C, dtype, fmt):
    x, g, _ = _case(R, C, R + C, dtype)
    dy = randn((R, C), R, dtype=dtype)
    mu, rs = _stats(x)
    m, r = mu[:, 0].float().to(DEV), rs[:, 0].float().to(DEV)
    xd, ck, kx = x.to(DEV), None, x
    if fmt != "none":
        ck, codes, scale = new_ckpt(R, C, fmt, 64)
        aqfq.aqfq_ckpt8_pack(ck, xd)
        torch.cuda.synchronize()
        kx, xd = kept(codes, scale, fmt, 64), None
    need = aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C)
    buf = torch.empty(need + 64, dtype=torch.uint8, device=DEV)
    first = None
    for off in (0, 8, 16, 24):
        buf.fill_(0xA5)
        dx, dg, db = torch.empty(R, C, dtype=dtype, device=DEV), *torch.empty(2, C, device=DEV)
        aqfq.aqfq_layernorm_bwd(dy.to(DEV), xd, m, r, g.to(DEV), dx, dgamma=dg, dbeta=db, ckpt=ck,
                                workspace=buf[off:off + need])
        torch.cuda.synchronize()
        assert bool((buf[:off] == 0xA5).all()) and bool((buf[off + need:] == 0xA5).all())
        if first is None:
            first = (dx, dg, db)
            _check_bwd(kx, dy, m, r, g, None, dx, dg, db)
        assert all(torch.equal(a, b) for a, b in zip(first, (dx, dg, db)))


# widths that fill their lanes and ones that leave some beyond the row, aligned and odd
@pytest.mark.parametrize("C", [8, 32, 64, 256, 512, 1024, 2048])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows_of_a_large_value(C, pad, dtype):
    """x - mean is zero all over the row: dx = rstd (dy gamma - mean(dy gamma)) and dgamma = 0
    though mean rstd is beyond binary32 (the widths are powers of two, so the mean is exact)."""
    R, big = 5, 1.5 * 2.0 ** 121
    rows = lambda t: torch.cat([t, torch.zeros(R, pad, dtype=t.dtype)], 1).to(DEV)[:, :C]
    x, dy = torch.full((R, C), big, dtype=dtype), randn((R, C), C, dtype=dtype)
    _, g, _ = _case(R, C, 5, dtype)
    m, r = torch.full((R,), big, device=DEV), torch.full((R,), 316.0, device=DEV)
    dx, dg, db = torch.empty(R, C, dtype=dtype, device=DEV), *torch.empty(2, C, device=DEV)
    w = torch.empty(aqfq.aqfq_layernorm_bwd_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
    aqfq.aqfq_layernorm_bwd(rows(dy), rows(x), m, r, g.to(DEV), dx, dgamma=dg, dbeta=db, workspace=w)
    torch.cuda.synchronize()
    _check_bwd(x, dy, m, r, g, None, dx, dg, db)
    assert bool((dg == 0).all())

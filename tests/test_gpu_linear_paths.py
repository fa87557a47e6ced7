"""The linear products where the kernel is chosen by the size, and operands as torch makes them.

Every test first asks which kernel its size takes.  Operands are small integers (times a power
of two), so that every sum is exact in any order: checkpoints and outputs without a smooth
activation are met bit for bit.  A smooth activation is at most E of its value, its derivative
E of its two terms off (test_gpu_activations.py); a stored BF16 value is rounded once more."""
import numpy as np
import pytest
import torch

from layerlib import ACTS, BF, DEV, U, close, grid_values, kept, new_ckpt, pack_ref, randn
from learnable_scale_fake_gb300 import aqfq
from test_gpu_activations import E, LEAST, terms, value64
from test_gpu_linear import ints, run_dgrad, run_fwd, run_wgrad

pytestmark = pytest.mark.gpu
FORMS = [("int8", 128), ("e4m3", 64), ("int8", 32), ("e4m3", 128)]


def product(a, b):
    """a @ b.T of operands whose sums are exact in binary32."""
    return (a.float().to(DEV) @ b.float().to(DEV).T).cpu()


def value(p, act):
    """act(p) in 64 bits and its error bound."""
    if act in ("none", "relu"):
        return (p if act == "none" else torch.clamp(p, min=0)).double(), torch.zeros(1).double()
    v = value64(p, act)
    return v, E * v.abs() + LEAST * (1 + p.abs())


def slope(p, act):
    if act in ("none", "relu"):
        return (torch.ones_like(p) if act == "none" else (p > 0)).double(), torch.zeros(1).double()
    a, b, amp = terms(p, act)
    return a + b, E * (a.abs() + b.abs()) + LEAST * amp


def check_fwd(M, N, K, act, form, with_res, seed=0, div=8.0):
    x, w = ints((M, K), 1 + seed, 1), ints((N, K), 2 + seed, 1) / div
    bias = ints((N,), 3) / 4.0
    res = randn((M, N), 4) if with_res else None
    fmt, group = form or (None, 0)
    y, codes, scale = run_fwd(x, w, bias, act, res, fmt, group, seed=seed)
    p = product(x, w) + bias.float()
    ref, e = value(p, act)
    if res is not None:
        ref = ref + res.double()
    close(y, ref, e + 2 * U * ref.abs() + BF * ref.abs(), act)
    if fmt:
        q, s = pack_ref(p, fmt, group)
        np.testing.assert_array_equal(scale.cpu().numpy(), s)
        np.testing.assert_array_equal(grid_values(codes, fmt), q)


def check_dgrad(M, N, K, act, form, with_res, seed=0, div=8.0):
    dy, w = ints((M, N), 5 + seed, 1), ints((N, K), 6 + seed, 1) / div
    res = randn((M, K), 7) if with_res else None
    fmt, group = form
    ck, codes, scale = new_ckpt(M, K, fmt, group)
    aqfq.aqfq_ckpt8_pack(ck, randn((M, K), 8, 1.5).to(DEV))
    dx = run_dgrad(dy, w, act, ck, res, seed=seed)
    a = product(dy, w.T).double()
    d, e = slope(kept(codes, scale, fmt, group), act)
    ref = a * d
    tol = a.abs() * e + 2 * U * ref.abs()
    if res is not None:
        ref = ref + res.double()
    close(dx, ref, tol + 2 * U * ref.abs() + BF * ref.abs(), act)


def check_wgrad(N, K, M, dtype, accumulate, seed=0):
    dy, x = ints((M, N), 9 + seed, 1), ints((M, K), 10 + seed, 1)
    base = ints((N, K), 11).to(dtype) if accumulate else None
    dw = run_wgrad(dy, x, dtype, base, seed=seed)
    ref = product(dy.T, x.T)
    if accumulate:
        ref = ref + base.float()
    assert torch.equal(dw.cpu(), ref.to(dtype))


# more than 152 tiles of 128 x 128: whole aligned blocks, ragged ones, an odd number of tile rows
ON_PAIRS = [(2048, 2560, 264), (2050, 2568, 200), (2303, 2509, 136)]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("form", [None] + FORMS)
def test_forward_on_pairs(act, form):
    for i, (M, N, K) in enumerate(ON_PAIRS):
        plan = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_FWD, M, N, K)
        assert plan == {"kernel": "pair", "splits": 1, "tail": 0, "tail_splits": 0}
        for with_res in ((False, True) if i == 0 else (i == 1,)):
            check_fwd(M, N, K, act, form, with_res, seed=i)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("form", FORMS)
def test_input_gradient_on_pairs(act, form):
    for i, (M, K, N) in enumerate(ON_PAIRS):
        plan = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_DGRAD, M, N, K)
        assert plan == {"kernel": "pair", "splits": 1, "tail": 0, "tail_splits": 0}
        for with_res in ((False, True) if i == 0 else (i == 1,)):
            check_dgrad(M, N, K, act, form, with_res, seed=i)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_on_pairs(dtype, accumulate):
    for i, (N, K, M) in enumerate(ON_PAIRS):
        assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_WGRAD, M, N, K)["kernel"] == "pair"
        check_wgrad(N, K, M, dtype, accumulate, seed=i)


# rows, columns, inner axis of outputs whose last tiles a second launch splits into 2 to 8
# slices; the same a little smaller in every axis
TAILS = [(1792, 2816, 3840, 8), (1536, 3584, 4096, 6), (1280, 4352, 4096, 5), (1280, 4608, 4352, 4),
         (5888, 1024, 4864, 3), (1280, 5120, 6656, 2)]
TAILS += [(r - 5, c - 11, d - 24, n) for r, c, d, n in TAILS]


@pytest.mark.parametrize("rows,cols,depth,cut", TAILS)
@pytest.mark.parametrize("kind", ["fwd", "dgrad", "wgrad"])
def test_last_tiles_split_by_a_second_launch(rows, cols, depth, cut, kind):
    i = [t[:3] for t in TAILS].index((rows, cols, depth))
    form, act = FORMS[i % 4], ["gelu", "relu", "silu", "none", "gelu_tanh"][i % 5]
    if kind == "fwd":
        plan = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_FWD, rows, cols, depth)
    elif kind == "dgrad":
        plan = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_DGRAD, rows, depth, cols)
    else:
        plan = aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_WGRAD, depth, rows, cols)
    assert plan["kernel"] == "pair" and plan["tail"] > 0 and plan["tail_splits"] == cut
    if kind == "fwd":
        check_fwd(rows, cols, depth, act, form, i % 2 == 0, seed=i % 3, div=64.0)
    elif kind == "dgrad":
        check_dgrad(rows, depth, cols, act, form, i % 2 == 0, seed=i % 3, div=64.0)
    else:
        check_wgrad(rows, cols, depth, torch.float32 if i % 2 else torch.bfloat16, i % 3 == 0, seed=i % 3)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_smooth_activations_through_scratch(act):
    """Sums in slices through scratch, the epilogue in a second kernel."""
    r, c, d = 70, 300, 33000
    assert aqfq.aqfq_selftest_linear_plan(aqfq.LINEAR_FWD, r, c, d)["splits"] > 1
    assert aqfq.aqfq_linear_workspace_bytes(aqfq.LINEAR_FWD, r, c, d) > 0
    check_fwd(r, c, d, act, FORMS[0], True, div=128.0)
    check_dgrad(r, d, c, act, FORMS[1], False, div=128.0)


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

"""The binding's calls between a layer's quantized products take tensors of one device, the
current one, and of the types and shapes that they document (stand-ins for tensors; nothing is
launched)."""
import pytest
import torch

from learnable_scale_fake_gb300 import aqfq
from test_layer_devices import BF, FL, I32, T, ck, fake, m, v  # noqa: F401 (fake: a fixture)


class H(T):
    """Heads [T, heads, D]."""

    def stride(self):
        return (self.shape[1] * self.shape[2], self.shape[2], 1)


def heads(n):
    return lambda dev=0, dtype=BF: H(8, n, 64, dtype=dtype, dev=dev)


# each call with every tensor it takes
CALLS = {
    "aqfq_rotary": lambda t: dict(
        q=t("q", heads(4)), yq=t("yq", heads(4)), k=t("k", heads(2)), yk=t("yk", heads(2)),
        pos=t("pos", lambda dev: v(8, torch.int64, dev)), freqs=t("freqs", lambda dev: v(32, torch.float64, dev))),
    "aqfq_block_norm_fwd": lambda t: dict(
        x=t("x", m), f=t("f", m), eps=1e-6, h=t("h", m), y=t("y", m), post=True,
        gamma_post=t("gamma_post", lambda dev: v(64, BF, dev)), gate=t("gate", lambda dev: v(64, BF, dev)),
        gamma_pre=t("gamma_pre", lambda dev: v(64, BF, dev)), rstd_post=t("rstd_post", lambda dev: v(8, FL, dev)),
        rstd_pre=t("rstd_pre", lambda dev: v(8, FL, dev))),
    "aqfq_block_norm_bwd": lambda t: dict(
        dy=t("dy", m), dh=t("dh", m), h=t("h", m), f=t("f", m), rstd_post=t("rstd_post", lambda dev: v(8, FL, dev)),
        rstd_pre=t("rstd_pre", lambda dev: v(8, FL, dev)), gamma_post=t("gamma_post", lambda dev: v(64, BF, dev)),
        gate=t("gate", lambda dev: v(64, BF, dev)), gamma_pre=t("gamma_pre", lambda dev: v(64, BF, dev)),
        dx=t("dx", m), df=t("df", m), dgamma_post=t("dgamma_post", lambda dev: v(64, FL, dev)),
        dgate=t("dgate", lambda dev: v(64, FL, dev)), dgamma_pre=t("dgamma_pre", lambda dev: v(64, FL, dev)),
        workspace=t("workspace", lambda dev: v(4, FL, dev))),
    "aqfq_gated_fwd": lambda t: dict(
        x=t("x", m), w=t("w", lambda dev: m(dev, 128, 64)), y=t("y", m), gate=t("gate", ck), up=t("up", ck),
        workspace=t("workspace", lambda dev: v(4, FL, dev)), error_flag=t("error_flag", lambda dev: v(1, I32, dev))),
    "aqfq_gated_dgrad": lambda t: dict(
        dy=t("dy", lambda dev: m(dev, 8, 48)), w=t("w", lambda dev: m(dev, 48, 64)),
        dp=t("dp", lambda dev: m(dev, 8, 128)), gate=t("gate", ck), up=t("up", ck), y=t("y", m),
        workspace=t("workspace", lambda dev: v(4, FL, dev)), error_flag=t("error_flag", lambda dev: v(1, I32, dev))),
    "aqfq_ckpt8_gated_bwd": lambda t: dict(
        gate=t("gate", ck), up=t("up", ck), act=aqfq.ACT_SILU, dy=t("dy", m), dp=t("dp", lambda dev: m(dev, 8, 128)),
        y=t("y", m)),
}


def names(call):
    seen = []
    CALLS[call](lambda name, make: seen.append(name))
    return seen


@pytest.mark.parametrize("call,other", [(c, n) for c in CALLS for n in names(c)])
def test_a_tensor_of_another_device_is_refused(fake, call, other):  # noqa: F811
    with pytest.raises(ValueError, match="cuda:1"):
        getattr(aqfq, call)(**CALLS[call](lambda name, make: make(dev=1 if name == other else 0)))
    assert not fake.calls


@pytest.mark.parametrize("call", list(CALLS))
def test_tensors_have_to_be_on_the_current_device(fake, call):  # noqa: F811
    getattr(aqfq, call)(**CALLS[call](lambda name, make: make(dev=0)))
    assert fake.calls == [call]
    with pytest.raises(ValueError, match="current device is cuda:0"):
        getattr(aqfq, call)(**CALLS[call](lambda name, make: make(dev=1)))
    assert fake.calls == [call]


def with_(call, **kw):
    a = CALLS[call](lambda name, make: make(dev=0))
    a.update(kw)
    return getattr(aqfq, call)(**a)


def test_types_and_shapes(fake):  # noqa: F811
    with pytest.raises(TypeError, match="yk"):
        with_("aqfq_rotary", yk=heads(2)(dtype=FL))
    with pytest.raises(TypeError, match="pos"):
        with_("aqfq_rotary", pos=v(8, I32))
    with pytest.raises(TypeError, match="freqs"):
        with_("aqfq_rotary", freqs=v(32, FL))
    with pytest.raises(ValueError, match="pos"):
        with_("aqfq_rotary", pos=v(7, torch.int64))
    with pytest.raises(ValueError, match="yk"):
        with_("aqfq_rotary", yk=heads(3)())
    with pytest.raises(ValueError, match="together"):
        with_("aqfq_rotary", k=None)
    with pytest.raises(ValueError, match="together"):
        with_("aqfq_rotary", yk=None)
    with pytest.raises(TypeError, match="one type"):
        with_("aqfq_block_norm_fwd", gate=v(64, FL))
    with pytest.raises(TypeError, match="one type"):
        with_("aqfq_block_norm_bwd", gamma_pre=v(64, FL))
    with pytest.raises(TypeError, match="f must"):
        with_("aqfq_block_norm_fwd", f=T(8, 64, dtype=FL))
    with pytest.raises(ValueError, match="rstd_pre"):
        with_("aqfq_block_norm_fwd", rstd_pre=v(7))
    with pytest.raises(ValueError, match="h must"):
        with_("aqfq_block_norm_bwd", h=m(0, 8, 32))
    with pytest.raises(TypeError, match="dgate"):
        with_("aqfq_block_norm_bwd", dgate=v(64, BF))
    with pytest.raises(ValueError, match="w must"):
        with_("aqfq_gated_fwd", w=m(0, 64, 64))
    with pytest.raises(ValueError, match="dp must"):
        with_("aqfq_gated_dgrad", dp=m(0, 8, 64))
    with pytest.raises(ValueError, match="checkpoint"):
        with_("aqfq_gated_dgrad", up=ck(0, 8, 32))
    with pytest.raises(TypeError, match="y must"):
        with_("aqfq_ckpt8_gated_bwd", y=T(8, 64, dtype=FL))
    assert not fake.calls

"""The binding's layer calls take tensors of one device, the current one (stand-ins for tensors
of two devices; nothing is launched)."""
import pytest
import torch

from learnable_scale_fake_gb300 import aqfq

BF, FL, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class T:
    """What the binding asks a tensor."""

    def __init__(self, *shape, dtype=BF, dev=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        self.is_cuda, self.nbytes = True, 1 << 30

    def get_device(self):
        return self.dev

    def stride(self):
        return (self.shape[1], 1)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class NoLaunch:
    """In the library's place: records what would have been called."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture()
def fake(monkeypatch):
    L = NoLaunch()
    monkeypatch.setattr(aqfq, "_lib", L)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(aqfq, "_raw_stream", lambda dev: 0)
    return L


def ck(dev=0, rows=8, cols=64):
    return aqfq.ckpt8(aqfq.INT8, 32, T(rows, cols, dtype=U8, dev=dev), T(rows, cols // 32, dtype=FL, dev=dev))


def m(dev=0, rows=8, cols=64):
    return T(rows, cols, dev=dev)


def v(n, dtype=FL, dev=0):
    return T(n, dtype=dtype, dev=dev)


# each call with every tensor it takes; W [48, 64], x [8, 64], dy of the products [8, 48]
CALLS = {
    "aqfq_ckpt8_pack": lambda t: dict(ckpt=t("ckpt", ck), x=t("x", m)),
    "aqfq_ckpt8_unpack": lambda t: dict(ckpt=t("ckpt", ck), y=t("y", m)),
    "aqfq_ckpt8_act_bwd": lambda t: dict(
        ckpt=t("ckpt", ck), act=aqfq.ACT_SILU, dy=t("dy", m), dx=t("dx", m), y=t("y", m),
        dbias=t("dbias", lambda dev: v(64, dev=dev)), workspace=t("workspace", lambda dev: v(4, dev=dev))),
    "aqfq_layernorm_fwd": lambda t: dict(
        x=t("x", m), gamma=t("gamma", lambda dev: v(64, BF, dev)), beta=t("beta", lambda dev: v(64, BF, dev)),
        eps=1e-5, y=t("y", m), mean=t("mean", lambda dev: v(8, dev=dev)),
        rstd=t("rstd", lambda dev: v(8, dev=dev)), ckpt=t("ckpt", ck)),
    "aqfq_layernorm_bwd": lambda t: dict(
        dy=t("dy", m), x=t("x", m), mean=t("mean", lambda dev: v(8, dev=dev)),
        rstd=t("rstd", lambda dev: v(8, dev=dev)), gamma=t("gamma", lambda dev: v(64, BF, dev)),
        dx=t("dx", m), dgamma=t("dgamma", lambda dev: v(64, dev=dev)),
        dbeta=t("dbeta", lambda dev: v(64, dev=dev)), dres=t("dres", m), ckpt=t("ckpt", ck),
        workspace=t("workspace", lambda dev: v(4, dev=dev))),
    "aqfq_linear_fwd": lambda t: dict(
        x=t("x", m), w=t("w", lambda dev: m(dev, 48, 64)), y=t("y", lambda dev: m(dev, 8, 48)),
        bias=t("bias", lambda dev: v(48, BF, dev)), residual=t("residual", lambda dev: m(dev, 8, 48)),
        workspace=t("workspace", lambda dev: v(4, dev=dev)),
        error_flag=t("error_flag", lambda dev: v(1, I32, dev))),
    "aqfq_linear_dgrad": lambda t: dict(
        dy=t("dy", lambda dev: m(dev, 8, 48)), w=t("w", lambda dev: m(dev, 48, 64)), dx=t("dx", m),
        act=aqfq.ACT_GELU, ckpt=t("ckpt", ck), residual=t("residual", m),
        workspace=t("workspace", lambda dev: v(4, dev=dev)),
        error_flag=t("error_flag", lambda dev: v(1, I32, dev))),
    "aqfq_linear_wgrad": lambda t: dict(
        dy=t("dy", lambda dev: m(dev, 8, 48)), x=t("x", m), dw=t("dw", lambda dev: m(dev, 48, 64)),
        workspace=t("workspace", lambda dev: v(4, dev=dev)),
        error_flag=t("error_flag", lambda dev: v(1, I32, dev))),
}


def names(call):
    seen = []
    CALLS[call](lambda name, make: seen.append(name))
    return seen


@pytest.mark.parametrize("call,other", [(c, n) for c in CALLS for n in names(c)])
def test_a_tensor_of_another_device_is_refused(fake, call, other):
    with pytest.raises(ValueError, match="cuda:1"):
        getattr(aqfq, call)(**CALLS[call](lambda name, make: make(dev=1 if name == other else 0)))
    assert not fake.calls


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("stream", [None, T])
def test_tensors_have_to_be_on_the_current_device(fake, call, stream):
    if stream is not None:
        stream = type("Stream", (), {"cuda_stream": 0})()
    getattr(aqfq, call)(**CALLS[call](lambda name, make: make(dev=0)), stream=stream)
    assert fake.calls == [call]
    with pytest.raises(ValueError, match="current device is cuda:0"):
        getattr(aqfq, call)(**CALLS[call](lambda name, make: make(dev=1)), stream=stream)
    assert fake.calls == [call]


def test_a_checkpoint_is_on_one_device():
    with pytest.raises(ValueError, match="cuda:1"):
        aqfq.ckpt8(aqfq.INT8, 32, T(8, 64, dtype=U8), T(8, 2, dtype=FL, dev=1))

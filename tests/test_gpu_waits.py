"""The bounded waits of the product kernels, from a small program around the same header."""
import ctypes
import os
import subprocess

import pytest
import torch

from learnable_scale_fake_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("waits") / "waits.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "device_waits.cu")
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-I", _build.CSRC, "-I", _build.INCLUDE,
                    "-shared", "-cudart", "shared", "-o", lib, src], check=True)
    return ctypes.CDLL(lib)


def test_a_warp_gives_up_as_one(waits):
    """Lanes with limits below and above the time the phase completes: alone some give up and
    some do not; the warp's answer is the same in every lane."""
    own, every = torch.full((2, 32), -1, dtype=torch.int32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    torch.cuda.synchronize()
    # limits of 1 to 32 units of 4 ms: well above the time a suspended try may take
    assert waits.run_uneven_limits(ctypes.c_longlong(1 << 23), p(own), p(every)) == 0
    own, every = own.cpu().tolist(), every.cpu().tolist()
    assert own[0] == 0 and own[31] == 1
    assert every == [0] * 32


@pytest.mark.parametrize("missing", [0, 1])
def test_drain_waits_for_the_loads_in_flight_and_no_longer_than_its_limit(waits, missing):
    src = torch.randint(0, 256, (5, 1024), dtype=torch.uint8, device="cuda")
    out, done = torch.zeros(3, 1024, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    torch.cuda.synchronize()
    assert waits.run_drain(p(src), missing, ctypes.c_longlong(1 << 22), p(out), p(done)) == 0
    assert int(done.item()) == 1
    # stages 0 and 1 hold loads 3 and 4, stage 2 load 2 (the announced sixth never arrives)
    assert torch.equal(out, src[[3, 4, 2]])


@pytest.mark.parametrize("turns,lost", [(7, 7), (7, 6), (7, 4), (2, 1), (7, 0)])
def test_ring_drains_what_is_on_its_way(waits, turns, lost):
    """A ring whose loads stop coming at turn `lost`: it gives up there, drains within its limits
    and returns; what was loaded before is in place."""
    src = torch.randint(0, 256, (7, 1024), dtype=torch.uint8, device="cuda")
    out, done = torch.zeros(3, 1024, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    torch.cuda.synchronize()
    assert waits.run_ring(p(src), turns, lost, ctypes.c_longlong(1 << 22), p(out), p(done)) == 0
    assert int(done.item()) == lost
    for i in range(max(0, lost - 3), lost):
        assert torch.equal(out[i % 3], src[i])

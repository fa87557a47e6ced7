"""Host logic of the library that needs no GPU."""
import os
import shutil
import subprocess

import pytest

from learnable_scale_fake_gb300 import _build, aqfq
from test_layer_sources import sources

ONCE = r"""
#include <cstdio>
#include "aqfq_once.h"
int main() {
  static aqfq::DeviceOnce once;
  int calls = 0, fail = 0;
  auto set = [&] { ++calls; return fail; };
  // the first call on each device sets, later ones do not
  if (once.run(0, set) || once.run(0, set) || calls != 1) return 1;
  if (once.run(1, set) || calls != 2) return 2;
  if (once.run(0, set) || once.run(1, set) || calls != 2) return 3;
  // a failure is reported and not kept
  fail = 7;
  if (once.run(2, set) != 7 || calls != 3 || once.run(2, set) != 7 || calls != 4) return 4;
  fail = 0;
  if (once.run(2, set) || once.run(2, set) || calls != 5) return 5;
  // an ordinal out of range is never remembered
  if (once.run(-1, set) || once.run(-1, set) || once.run(256, set) || calls != 8) return 6;
  return 0;
}
"""


def test_a_kernels_attributes_are_set_once_per_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(ONCE)
    subprocess.run([cxx, "-std=c++17", "-I", _build.CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_no_kernel_sets_its_attributes_once_per_process():
    for f, s in sources().items():
        at = s.find("cudaFuncSetAttribute")
        while at >= 0:
            # the statement that the call is part of
            start = max(s.rfind(c, 0, at) for c in ";{}")
            assert "static" not in s[start:at], f
            at = s.find("cudaFuncSetAttribute", at + 1)
        assert not ("call_once" in s and "cudaFuncSetAttribute" in s.split("call_once", 1)[1][:300]), f
    assert os.path.exists(os.path.join(_build.CSRC, "aqfq_once.h"))


def test_operands_without_elements_need_no_alignment():
    """A contiguous [rows, 0] tensor has rows one element apart; nothing is launched here."""
    _build.build()
    L, A = aqfq.lib(), 0x10000
    assert L.aqfq_linear_fwd(None, 1, None, 1, 0, 5, 0, 0, None, 0, None, 0, None, 8, None, None, 0, None, None) == 0
    assert L.aqfq_linear_dgrad(A, 8, A + 2, 1, 4, 5, 0, 0, None, None, 0, None, 1, None, 0, None, None) == 0
    assert L.aqfq_linear_wgrad(A, 8, A + 2, 1, 4, 5, 0, 0, None, 1, 0, None, 0, None, None) == 0
    # with elements the rule stands
    assert L.aqfq_linear_fwd(A, 9, A, 16, 4, 5, 9, 0, None, 0, None, 0, A, 8, None, None, 0, None, None) == 3

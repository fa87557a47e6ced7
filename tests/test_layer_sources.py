"""Rules that the kernels' sources have to keep, read from the sources (no GPU)."""
import os
import re

from learnable_scale_fake_gb300 import _build


def sources():
    """file name -> source without comments, neighbouring string literals joined"""
    out = {}
    for f in sorted(os.listdir(_build.CSRC)):
        s = open(os.path.join(_build.CSRC, f)).read()
        s = re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)
        out[f] = re.sub(r'"\s*"', "", s)
    return out


def test_no_load_is_multicast_to_a_cluster():
    """Every rank of a multi-GPU launch loads this library, and a multicast load may read only
    memory of its own GPU, which an address does not show: no bulk copy has it.  (A tcgen05
    commit that signals barriers of several blocks moves no data.)"""
    found = {}
    for f, s in sources().items():
        for text in re.findall(r'"((?:[^"\\]|\\.)*)"', s):
            if "cp.async.bulk" in text and "multicast" in text:
                found[f] = text
    assert not found
    # the rule sees the copies that are there
    assert any("cp.async.bulk.tensor" in s for s in sources().values())

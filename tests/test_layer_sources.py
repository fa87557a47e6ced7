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


def test_waits_of_the_products_are_uniform_in_a_warp():
    """The product kernels' loops issue warp-wide instructions after a bounded wait: the answer
    has to be the warp's, or one thread's that hands it on."""
    s = sources()["aqfq_linear.cu"]
    alone = [m.start() for m in re.finditer(r"\bmbar_(?:wait|wait_long|wait_suspend)\(", s)]
    for at in alone:
        block = s[:at].rsplit("if (", 1)[1]
        assert re.match(r"warp == \d+ && lane == 0\)", block), s[at - 200:at + 80]
    assert len(re.findall(r"\bmbar_wait_warp\(", s)) >= 7


def test_products_drain_their_loads_before_a_block_ends():
    """After a wait that gave up, whichever it was: both kernels wait (bounded) for the loads in
    flight past their last barrier, before the block's memory goes to another one."""
    s = sources()["aqfq_linear.cu"]
    drain = r"if \(warp == 0 && (?:rank == 0 && )?\*abort\) drain_loads\(sh->full, \S+ sh->issued\);"
    assert len(re.findall(drain, s)) == 3
    assert len(re.findall(r"sh->issued = \w+;", s)) == 2

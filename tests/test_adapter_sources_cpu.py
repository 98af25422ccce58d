"""Rules of the adapters' kernels that no run can show, read from their sources: an instruction that wants a
converged warp (``.aligned``) is not left to the compiler's reconvergence behind code in which lanes part."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "int8_mixed_precision_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["adapters.cuh", "adapters.cu", "adapters_small.cu"])
def test_cluster_barriers_want_a_converged_warp(name):
    """The loop before a cluster's last barrier has unequal trip counts: with three CTAs and a rank of 16 the lanes
    of a warp leave the sum of h in different iterations."""
    text = code(name)
    for m in re.finditer(r'asm volatile\("barrier\.cluster[^"]*aligned', text):
        before = re.sub(r"if \(p\.cluster > 1\)\s*\{?\s*$", "", text[:m.start()].rstrip()).rstrip()
        assert before.endswith(("__syncwarp();", "__syncthreads();")), (name, text[m.start():m.start() + 60], before[-80:])


def test_lanes_are_back_from_an_arrival_before_the_next_panel_is_read():
    text = code("adapters.cu")
    loops = re.findall(r"for \(int i = 0; i < all; \+\+i\) \{(.*?)tmem_ld8", text, re.S)
    assert len(loops) == 1 and "__syncwarp();" in loops[0]

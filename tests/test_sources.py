"""The library's sources: what its kernels must not contain."""
import glob
import os
import re

import pytest

from gated_delta_rule_52_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu*")))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_no_multicast_loads(path):
    """No bulk or tensor load into several CTAs at once: the library is loaded by ranks that map other
    GPUs' memory too, and an operand's pointer may be to such memory.  (The multicast of a
    tcgen05.commit is an arrival on barriers and loads nothing.)"""
    text = open(path).read()
    assert not [i for i in re.findall(r"cp\.async\.bulk[\w.:]*", text) if "multicast" in i]

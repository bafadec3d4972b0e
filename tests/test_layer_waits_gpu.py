"""The scans' bounded waits run out and say so: the first one after its limit, those after it
at once, so that a kernel ends soon however many values or copies are missing."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_delta_rule_52_gb300 import build, kda

pytestmark = pytest.mark.gpu

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "csrc", "scan_waits.cu")
vp, ci = ctypes.c_void_p, ctypes.c_int


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("waits") / "libscan_waits.so")
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", out, SRC, "-lcuda"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    L = ctypes.CDLL(out)
    L.scan_value_waits.argtypes = [vp, vp, ci, vp, vp]
    L.scan_copy_waits.argtypes = [ci, vp, vp]
    return L


def _ms(call):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    assert call(torch.cuda.current_stream().cuda_stream) == 0
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


def test_missing_values(waits):
    n = 200
    empty = torch.full((3 * n,), -1, dtype=torch.int32, device="cuda")        # all ones: nothing published
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def ms(count):
        err.zero_()
        return _ms(lambda s: waits.scan_value_waits(empty.data_ptr(), empty.data_ptr() + 8 * n, count, err.data_ptr(), s))

    # one state and one map: a wait to its limit, below 10 s; 398 further ones take less than another
    first = ms(1)
    assert err.item() == kda.KDA_ERR_TIMEOUT and first < 10e3
    many = ms(n)
    assert err.item() == kda.KDA_ERR_TIMEOUT and many < 2 * first + 1e3, (first, many)


def test_published_values_are_not_waited_for(waits):
    n = 200
    there = torch.ones(3 * n, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ms = _ms(lambda s: waits.scan_value_waits(there.data_ptr(), there.data_ptr() + 8 * n, n, err.data_ptr(), s))
    assert err.item() == 0 and ms < 1e3


def test_missing_copies(waits):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # 2 s, then a millisecond each (and what a single try of the barrier takes)
    ms = _ms(lambda s: waits.scan_copy_waits(100, err.data_ptr(), s))
    assert err.item() == kda.KDA_ERR_TIMEOUT and 1.9e3 < ms < 4e3, ms

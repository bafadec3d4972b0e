"""The 8-bit product's bounded waits run out after their limit, for the whole warp, and not before."""
import ctypes
import os
import subprocess

import pytest
import torch

from gated_delta_rule_52_gb300 import build

pytestmark = pytest.mark.gpu

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "csrc", "product_waits.cu")


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("waits") / "libproduct_waits.so")
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", out, SRC, "-lcuda"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    L = ctypes.CDLL(out)
    L.product_wait.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]
    L.product_wait_limit.restype = ctypes.c_uint64
    for cluster in (0, 1):      # the first launch loads the kernels
        _wait(L, cluster, 1, 10 ** 6)
    return L


def _wait(waits, cluster, arrivals, limit):
    got = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    assert waits.product_wait(cluster, arrivals, limit, got.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    b.record()
    torch.cuda.synchronize()
    return got.tolist(), a.elapsed_time(b)


@pytest.mark.parametrize("cluster", [0, 1])
def test_a_barrier_that_nothing_arrives_on(waits, cluster):
    assert waits.product_wait_limit() == 2 * 10 ** 9
    got, ms = _wait(waits, cluster, 0, 200 * 10 ** 6)
    assert got == [0] * 32 and 199 < ms < 400, ms


@pytest.mark.parametrize("cluster", [0, 1])
def test_a_phase_that_is_complete(waits, cluster):
    got, ms = _wait(waits, cluster, 1, 200 * 10 ** 6)
    assert got == [1] * 32 and ms < 100, ms

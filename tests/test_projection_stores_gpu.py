"""The 8-bit product's tensor stores where tiles follow one another at once: a short K, several tiles to
a pair of SMs, an odd number of stores to a tile.  A store's buffer is not written again before the
store has read it: whole numbers, whose sums are exact, come out the same every time."""
import pytest
import torch

from gated_delta_rule_52_gb300 import fp8, kda
from tests import projection_ref as ref
from tests.projection_ref import E4
from tests.test_projection_ops_gpu import _gen, _small_operand

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32

SHAPES = [(8192, 8192), (16384, 1024), (8192, 1792)]
# the last columns end inside the first or second 64 bytes of a half, so that a ragged tile has one store
# or none, and rows inside a tile; rows of out are 16 bytes aligned
RAGGED = [(6150, 2312, F), (4999, 1924, F), (4999, 3096, BF), (6143, 2312, HF), (8192, 1544, BF)]


def _check(M, N, K, dt, add):
    g = _gen(M + N + K)
    a, sa = _small_operand(M, K, E4, False, g)
    b, sb = _small_operand(N, K, E4, True, g)
    plus = torch.randint(-8, 9, (M, N), generator=g).to(dt).cuda() if add else None
    outs = [torch.full((M, N), float("nan"), dtype=dt, device="cuda") for _ in range(3)]
    for _ in range(4):
        for o in outs:
            fp8.matmul(a, sa, b, sb, o, add=plus)
    torch.cuda.synchronize()
    assert kda.get_device_status() == kda.KDA_OK
    want = ref.product(a, sa, b, sb, plus).float().to(dt)
    for o in outs:
        assert torch.equal(o.cpu(), want)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("K", [128, 256])
@pytest.mark.parametrize("M,N", SHAPES)
def test_stores_of_many_tiles(M, N, K, dt):
    _check(M, N, K, dt, False)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("M,N,dt", RAGGED)
def test_stores_of_ragged_tiles(M, N, dt, add):
    _check(M, N, 128, dt, add)


# rows of out that begin at multiples of 16 bytes and end between them: part of a wider tensor
PARTS = [(65, 1, 5), (100, 5, 31), (221, 29, 55), (300, 37, 640), (152, 409, 172), (3194, 33, 2061), (1763, 2521, 55), (4999, 1927, 128), (8192, 1795, 256),
         (300, 67, 4100), (130, 6501, 4100), (40, 67, 300), (3, 1001, 128)]


@pytest.mark.parametrize("dt", [BF, HF, F])
@pytest.mark.parametrize("M,N,K", PARTS)
def test_stores_end_with_the_row(M, N, K, dt):
    """What lies behind a row's end stays as it is."""
    g = _gen(M + N + K)
    a, sa = _small_operand(M, K, E4, False, g)
    b, sb = _small_operand(N, K, E4, True, g)
    V = 16 // dt.itemsize
    product = ref.product(a, sa, b, sb)
    for lead, add in ((0, False), (V, True)):
        wide = torch.full((M, -(-(lead + N) // V) * V + V), 7.0, dtype=dt, device="cuda")
        out = wide[:, lead:lead + N]
        if add:
            out.copy_(torch.randint(-8, 9, (M, N), generator=g).to(dt))
        want = (product + out.cpu().double() if add else product).float().to(dt)
        for _ in range(2):
            if add:
                kept = out.clone()
            fp8.matmul(a, sa, b, sb, out, add=out if add else None)
            assert torch.equal(out.cpu(), want)
            assert (wide[:, :lead] == 7).all() and (wide[:, lead + N:] == 7).all()
            if add:
                out.copy_(kept)
    torch.cuda.synchronize()
    assert kda.get_device_status() == kda.KDA_OK

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

"""What 32-bit sums of the 8-bit product over a long K may be off.

The tensor cores cut an accumulator towards zero at each step, so the product takes K in segments of
8192 whose sums are added in registers.  The operands here have elements of 13 and 15 and scales of 1
and 1/16: every segment's sum is below 2^24 units of 1/16, which an accumulator holds exactly, while
two segments' is not.  What is left are the additions of segments, each off by half a step of the sum:
2^-24 of it.  A sum that stayed in an accumulator would lose half a unit or more at each of its MMAs
beyond 2^24 units, a hundred times what is allowed after one segment too many."""
import pytest
import torch

from gated_delta_rule_52_gb300 import fp8, kda
from tests.projection_ref import E4

pytestmark = pytest.mark.gpu

SEGMENT = 8192
F = torch.float32

# rows of a, rows of b, K: one kernel or another by the rows and the tiles, and of few rows by the
# segments; whole segments and ragged ones
CASES = [(1, 300, 16384), (3, 40, 65536), (3, 40, 131072), (16, 200, 300000), (3, 40, 983040), (2, 40, 983168), (5, 130, 1 << 20),
         (20, 40, 458752), (20, 129, 500000), (33, 256, 131072), (64, 40, 196608), (40, 136, 196736), (64, 264, 400001),
         (65, 100, 16384), (200, 260, 32768), (128, 300, 30000), (300, 520, 65536), (1100, 1800, 16400), (4999, 1033, 24576),
         (256, 8300, 20000)]


def _operand(rows, K, g):
    q, s = fp8.empty(rows, K, E4)
    q.copy_(torch.randint(0, 2, (rows, K), generator=g, device="cuda").float() * 2 + 13)
    # half of the blocks of every segment
    e = torch.full((rows, s.shape[1]), 127, dtype=torch.uint8, device="cuda")
    e[:, 1::2] = 123
    s.view(torch.uint8).copy_(e)
    return q, s


def _segment_sums(a, b, K):
    """The segments' sums, exact in units of 1/16: [segments, M, N] doubles.  The scales are a block's:
    (1/16)^2 in odd blocks would be too fine, so b has scales of 1."""
    out = []
    for k in range(0, K, SEGMENT):
        w = torch.ones(min(SEGMENT, K - k), dtype=torch.float64, device="cuda")
        w[(torch.arange(k, k + len(w), device="cuda") // 128) % 2 == 1] = 1 / 16
        out.append((a[:, k:k + SEGMENT].float().double() * w) @ b[:, k:k + SEGMENT].float().double().T)
    return torch.stack(out)


@pytest.mark.parametrize("M,N,K", CASES)
def test_sums_of_a_long_k(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, sa = _operand(M, K, g)
    b, sb = _operand(N, K, g)
    sb.view(torch.uint8).fill_(127)
    parts = _segment_sums(a, b, K)
    assert float(parts.max()) * 16 < 2 ** 24
    want = parts.sum(0)
    out = torch.full((M, N), float("nan"), device="cuda")
    fp8.matmul(a, sa, b, sb, out)
    torch.cuda.synchronize()
    assert kda.get_device_status() == kda.KDA_OK
    # each segment added once, and up to 8 parts of K joined
    off = (out.double() - want).abs() / want * 2 ** 24
    assert float(off.max()) <= len(parts) + 8


@pytest.mark.parametrize("M,N,K", [(64, 40, 400001), (20, 131, 500003), (1, 33, 2000000)])
@pytest.mark.parametrize("add", ["own", "row", "out"])
def test_addends_of_a_long_k(M, N, K, add):
    """A K that few rows take in pieces: the addend counts once, also in place.  Whole numbers, exact sums."""
    g = torch.Generator(device="cuda").manual_seed(K)
    a, sa, b, sb = *fp8.empty(M, K, E4), *fp8.empty(N, K, E4)
    for q, s in ((a, sa), (b, sb)):
        q.copy_(torch.randint(-3, 4, q.shape, generator=g, device="cuda").float())
        s.view(torch.uint8).fill_(127)
    out = torch.full((M, N), float("nan"), device="cuda")
    plus = torch.randint(-99, 100, (1 if add == "row" else M, N), generator=g, device="cuda").float().expand(M, N)
    want = a.float() @ b.float().T
    want = want.double() + plus.double()
    assert float(want.abs().max()) < 2 ** 20
    if add == "out":
        out.copy_(plus)
        plus = out
    fp8.matmul(a, sa, b, sb, out, add=plus)
    torch.cuda.synchronize()
    assert kda.get_device_status() == kda.KDA_OK
    assert torch.equal(out.double(), want)

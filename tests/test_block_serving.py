"""Serving hands the residual stream from block to block, in 8 bits or not, in any order."""
import itertools

import pytest
import torch

from gated_delta_rule_52_gb300 import block


class _Block:
    """Adds ``k`` times the stream's running sum over tokens, as a block does: at once, or in 8 bits by way
    of what the next block's norm adds."""

    def __init__(self, k, eight):
        self.k, self.eight = k, eight

    def state(self, B):
        return {"sum": torch.zeros(B, 1, 2, dtype=torch.float64)}

    def _mix(self, u, state):
        c = state["sum"] + u.cumsum(1)
        state["sum"] = c[:, -1:]
        return self.k * c

    def serve(self, u, state):
        return u + self._mix(u, state)

    def serve_eight(self, u, delta, state):
        if delta is not None:
            u += delta
        return self._mix(u, state)


@pytest.mark.parametrize("eight", list(itertools.product([False, True], repeat=3)))
def test_blocks_in_any_order(eight):
    u = torch.arange(20.0, dtype=torch.float64).view(2, 5, 2) - 7
    before, want = u.clone(), u
    for i in range(3):
        want = want + (i + 1) * want.cumsum(1)
    got = block.serve([_Block(i + 1, e) for i, e in enumerate(eight)], u, 3)
    assert torch.equal(got, want) and torch.equal(u, before)

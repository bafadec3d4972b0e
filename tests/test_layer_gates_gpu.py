"""Gradients of the gated linear recurrence where its gates are saturated: every element
within the bound that the 64-bit reference carries for it (tests/layer_ref.py)."""
import math

import pytest
import torch

from tests.layer_ref import assert_close
from tests.test_layer_ops_gpu import _gen, _glr_check, _glr_inputs, _glr_ref, _glr_run

pytestmark = pytest.mark.gpu

BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def _saturated(dt, lb, T=200, K=40):
    """Logits spread evenly over [-16, 16], the range that the reference's bounds are made
    for: there 1 - sigma is down to 1e-7, one unit of fp32 below 1.  The input gate's logit
    is i; the bounded gate's is exp(A_log) (g + dt_bias) with exp(A_log) = 16, the other's
    g + dt_bias, up to 8 as decays beyond e^-10 leave nothing to compare."""
    d = _glr_inputs(2, T, 2, K, dt, None, F, 31)
    g = _gen(32)
    even = lambda *s: torch.rand(s, generator=g) * 2 - 1  # noqa: E731
    d["dt_bias"] = 0.25 * even(2, K)
    d["i"] = (16 * even(2, T, 2, K)).to(dt)
    if lb is None:
        d["g"] = (12 * even(2, T, 2, K) - 4 - d["dt_bias"]).to(dt)
    else:
        d["A_log"] = torch.full((2,), math.log(16.0))
        d["g"] = (even(2, T, 2, K) - d["dt_bias"]).to(dt)
    d["dout"] = (d["dout"] * 16).to(dt)   # gradients of 1e-6 times it are no subnormal fp16 numbers
    return d


@pytest.mark.parametrize("how", ["dense", "odd"])
@pytest.mark.parametrize("lb", [-5.0, None])
@pytest.mark.parametrize("dt", [BF, HF, F])
def test_gradients_of_saturated_gates(dt, lb, how):
    d = _saturated(dt, lb)
    _glr_check(_glr_run(d, lb, how), _glr_ref(d, lb))


def test_parameter_gradients_of_tokens_whose_gates_are_open():
    # every bounded gate above 12: ddt_bias and dA_log, in 32 bits, are sums of terms in
    # 1 - sigma alone
    d = _saturated(BF, -5.0)
    d["g"] = (0.875 + 0.125 * torch.rand(d["g"].shape, generator=_gen(33)) - d["dt_bias"]).to(BF)
    got, want = _glr_run(d, -5.0), _glr_ref(d, -5.0)
    for name in ("dg", "ddt_bias", "dA_log"):
        assert_close(name, got[name], *want[name])

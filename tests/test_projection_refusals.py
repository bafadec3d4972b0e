"""Calls of the operators around a layer's projections that are refused before anything runs, without
a GPU and without stand-ins for one."""
import pytest
import torch

from gated_delta_rule_52_gb300 import fp8, rms_norm


def _calls():
    x, row = torch.zeros(4, 128), torch.zeros(4)
    q, s = fp8.empty(4, 128, device="cpu")
    return [lambda: fp8.quantize(x, q, s), lambda: fp8.quantize(x, qt=fp8.empty(128, 4, device="cpu")[0], scales_t=fp8.empty(128, 4, device="cpu")[1]),
            lambda: fp8.dequantize(q, s, x), lambda: fp8.matmul(q, s, q, s, torch.zeros(4, 4)),
            lambda: rms_norm.rms_norm_fwd(x, None, 1e-6, x), lambda: rms_norm.rms_norm_fwd(x, None, 1e-6, q, scales=s),
            lambda: rms_norm.rms_norm_bwd(x, x, None, row)]


@pytest.mark.parametrize("i", range(len(_calls())))
def test_tensors_of_the_host(i):
    """A ValueError that says so, as from the other operators, also where there is no GPU to ask about."""
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        _calls()[i]()

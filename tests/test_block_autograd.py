"""The example's autograd functions refuse a second derivative, which their kernels do not
have.  Without a GPU: the operators are replaced by ones that write and return zeros."""
import pytest
import torch

from gated_delta_rule_52_gb300 import block, glr, kda, layer_norm, short_conv

N = lambda *s: torch.randn(s, requires_grad=True)  # noqa: E731

CASES = {
    "Norm": lambda: (N(3, 8), N(8), N(8)),
    "Conv": lambda: (N(1, 5, 8), N(8, 4), N(8)),
    "Recurrence": lambda: (N(1, 5, 2, 4), N(1, 5, 2, 4), N(1, 5, 2, 4), N(2), N(2, 4)),
    "DeltaRule": lambda: (*(N(1, 5, 2, 4) for _ in range(4)), N(1, 5, 2), N(2), N(2, 4)),
}
GRADS = {"Norm": ("dx", "dweight", "dbias"), "Conv": ("dx", "dweight", "dbias"),
         "Recurrence": ("dx", "di", "dg", "dA_log", "ddt_bias"),
         "DeltaRule": ("dq", "dk", "dv", "dg", "dbeta", "dA_log", "ddt_bias")}
OPS = {"Norm": (layer_norm, "layer_norm"), "Conv": (short_conv, "short_conv"), "Recurrence": (glr, "glr"), "DeltaRule": (kda, "kda")}


@pytest.mark.parametrize("name", CASES)
def test_second_derivative_is_refused(name, monkeypatch):
    inputs = CASES[name]()
    module, op = OPS[name]
    grads = {k: torch.ones_like(t) for k, t in zip(GRADS[name], inputs)}
    monkeypatch.setattr(module, op + "_fwd", lambda *a, **k: None)
    monkeypatch.setattr(module, op + "_bwd", lambda *a, **k: grads)
    out = getattr(block, name).apply(*inputs)
    first = torch.autograd.grad(out.sum(), inputs, create_graph=True, retain_graph=True)
    for got, t in zip(first, inputs):
        assert torch.equal(got, torch.ones_like(t))
    with pytest.raises(RuntimeError, match="first derivative"):
        torch.autograd.grad((first[0].square() + inputs[0].square()).sum(), inputs[0])

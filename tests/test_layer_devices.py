"""Calls of the operators around the delta rule whose tensors or stream are not on the
current GPU are refused before a pointer reaches the library.  Without a GPU: CPU tensors
that say where they are, and an entry point that notes that it was called."""
import pytest
import torch

from gated_delta_rule_52_gb300 import _args, glr, layer_norm, short_conv

F, BF, I = torch.float32, torch.bfloat16, torch.int64


class _OnGpu(torch.Tensor):
    is_cuda = True
    gpu = 0

    def get_device(self):
        return self.gpu


class _Stream:
    cuda_stream = 0

    def __init__(self, index):
        self.device_index = index


def _t(*shape, dtype=F):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


def _glr():
    u = lambda: _t(1, 6, 2, 8, dtype=BF)  # noqa: E731
    return {"x": u(), "i": u(), "g": u(), "A_log": _t(2), "dt_bias": _t(2, 8), "initial_state": _t(2, 2, 8),
            "cu_seqlens": _t(3, dtype=I), "checkpoints": _t(1, 2, 8), "lower_bound": -5.0, "stream": _Stream(0)}


def _conv():
    return {"x": _t(1, 6, 8, dtype=BF), "weight": _t(8, 4), "bias": _t(8), "initial_state": _t(2, 3, 8, dtype=BF),
            "cu_seqlens": _t(3, dtype=I), "stream": _Stream(0)}


CALLS = {
    "glr_fwd": (glr.glr_fwd, lambda: {**_glr(), "out": _t(1, 6, 2, 8, dtype=BF), "final_state": _t(2, 2, 8)}),
    "glr_bwd": (glr.glr_bwd, lambda: {**_glr(), "dout": _t(1, 6, 2, 8, dtype=BF), "dfinal": _t(2, 2, 8)}),
    "layer_norm_fwd": (layer_norm.layer_norm_fwd, lambda: {
        "x": _t(6, 8), "weight": _t(8), "bias": _t(8), "eps": 1e-5, "out": _t(6, 8), "mean": _t(6), "rstd": _t(6), "stream": _Stream(0)}),
    "layer_norm_bwd": (layer_norm.layer_norm_bwd, lambda: {
        "dout": _t(6, 8), "x": _t(6, 8), "weight": _t(8), "mean": _t(6), "rstd": _t(6), "stream": _Stream(0)}),
    "short_conv_fwd": (short_conv.short_conv_fwd, lambda: {**_conv(), "out": _t(1, 6, 8, dtype=BF), "final_state": _t(2, 3, 8, dtype=BF)}),
    "short_conv_bwd": (short_conv.short_conv_bwd, lambda: {**_conv(), "dout": _t(1, 6, 8, dtype=BF), "dfinal": _t(2, 3, 8)}),
}


@pytest.fixture
def calls(monkeypatch):
    """The entry points' calls, and the current GPU (a one-entry list)."""
    made, current = [], [0]
    monkeypatch.setattr(_args, "entry", lambda name: lambda *a: made.append(name) or 0)
    monkeypatch.setattr(_args, "current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(_args, "new", lambda stream, t, *shapes: [None if s is None else _t(*s, dtype=t.dtype) for s in shapes])
    return made, current


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_and_the_stream_on_the_current_gpu(name, calls):
    made, current = calls
    call, arguments = CALLS[name]
    call(**arguments())
    assert made == ["kda_" + name]
    made.clear()
    for k, v in arguments().items():
        if not isinstance(v, (torch.Tensor, _Stream)):
            continue
        a = arguments()
        if k == "stream":
            a[k] = _Stream(1)
        else:
            a[k].gpu = 1
        with pytest.raises(ValueError, match="cuda:1"):
            call(**a)
        assert not made, k
    current[0] = 1                      # all of them elsewhere
    with pytest.raises(ValueError, match="cuda:1"):
        call(**arguments())
    assert not made
    a = arguments()
    for k, v in a.items():
        if isinstance(v, torch.Tensor):
            v.gpu = 1
    a["stream"] = _Stream(1)
    call(**a)
    assert made == ["kda_" + name]

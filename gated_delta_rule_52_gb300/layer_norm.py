"""Layer norm over the last axis, forward and backward (C entry points
kda_layer_norm_fwd and kda_layer_norm_bwd of include/kda.h):

    out = (x - mean) * rstd * weight + bias,   rstd = 1 / sqrt(variance + eps)

``x`` is [..., D] in bf16, fp16 or fp32, rows evenly spaced (a slice of a wider tensor
qualifies); ``weight`` and ``bias`` are fp32 [D] or None; statistics are fp32.
"""
from __future__ import annotations

import torch

from . import _args, kda


def _shape(x):
    dt = _args.dtype_code("x", x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    n = 1
    for s in x.shape[:-1]:
        n *= s
    return dt, n, x.shape[-1], _args.rows("x", x, x.dtype, x.shape, x.dim() - 1)


def layer_norm_fwd(x, weight, bias, eps, out, mean=None, rstd=None, stream=None) -> None:
    """Writes ``out`` (like ``x``, and may be ``x``) and, where given, ``mean`` and ``rstd``
    (fp32, one value per row), asynchronously on ``stream`` (default: the current torch
    stream)."""
    dt, n, D, stride = _shape(x)
    out_stride = _args.rows("out", out, x.dtype, x.shape, x.dim() - 1)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _args.check(name, t, torch.float32, (D,))
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _args.check(name, t, torch.float32, x.shape[:-1])
    p = _args.ptr
    _args.done(kda.lib().kda_layer_norm_fwd(p(x), stride, p(weight), p(bias), eps, p(out), out_stride, p(mean),
                                            p(rstd), dt, n, D, _args.stream_handle(stream)))


def layer_norm_bwd(dout, x, weight, mean, rstd, want_params=None, stream=None) -> dict:
    """Gradients of sum(dout * out), with ``mean`` and ``rstd`` as the forward wrote them.
    Returns a dict of new tensors: dx (like x, contiguous), and fp32 dweight and dbias
    (None unless ``want_params``, by default where there is a weight)."""
    dt, n, D, stride = _shape(x)
    dout_stride = _args.rows("dout", dout, x.dtype, x.shape, x.dim() - 1)
    if weight is not None:
        _args.check("weight", weight, torch.float32, (D,))
    for name, t in (("mean", mean), ("rstd", rstd)):
        _args.check(name, t, torch.float32, x.shape[:-1])
    if want_params is None:
        want_params = weight is not None
    with _args.on(stream):
        r = {"dx": torch.empty(x.shape, dtype=x.dtype, device=x.device), "dweight": None, "dbias": None}
        if want_params:
            r["dweight"] = torch.empty((D,), dtype=torch.float32, device=x.device)
            r["dbias"] = torch.empty((D,), dtype=torch.float32, device=x.device)
    p = _args.ptr
    _args.done(kda.lib().kda_layer_norm_bwd(p(dout), dout_stride, p(x), stride, p(weight), p(mean), p(rstd),
                                            p(r["dx"]), p(r["dweight"]), p(r["dbias"]), dt, n, D,
                                            _args.stream_handle(stream)))
    return r

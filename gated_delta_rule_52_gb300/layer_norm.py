"""Layer norm over the last axis, forward and backward (C entry points
kda_layer_norm_fwd and kda_layer_norm_bwd of include/kda.h):

    out = (x - mean) * rstd * weight + bias,   rstd = 1 / sqrt(variance + eps)

``x`` is [..., D] in bf16, fp16 or fp32, rows evenly spaced (a slice of a wider tensor
qualifies); ``weight`` and ``bias`` are fp32 [D] or None; statistics are fp32.
"""
from __future__ import annotations

import math

import torch

from . import _args


def _shape(x):
    dt, shape = _args.dtype_code("x", x), x.shape
    if not shape:
        raise ValueError("x must have at least one dimension")
    D, lead, dev = shape[-1], len(shape) - 1, _args.device("x", x)
    return dev, dt, shape, lead, D, _args.rows("x", x, x.dtype, shape, lead, D, dev)


def layer_norm_fwd(x, weight, bias, eps, out, mean=None, rstd=None, stream=None) -> None:
    """Writes ``out`` (like ``x``, and may be ``x``) and, where given, ``mean`` and ``rstd``
    (fp32, one value per row), asynchronously on ``stream`` (default: the current torch
    stream)."""
    dev, dt, shape, lead, D, stride = _shape(x)
    out_stride = _args.rows("out", out, x.dtype, shape, lead, D, dev)
    f32, row, param = torch.float32, shape[:-1], (D,)
    _args.done(_args.entry("kda_layer_norm_fwd")(
        x.data_ptr(), stride, _args.optional("weight", weight, f32, param, dev), _args.optional("bias", bias, f32, param, dev), eps,
        out.data_ptr(), out_stride, _args.optional("mean", mean, f32, row, dev), _args.optional("rstd", rstd, f32, row, dev), dt,
        math.prod(row), D, _args.stream_handle(stream, dev)))


def layer_norm_bwd(dout, x, weight, mean, rstd, want_params=None, stream=None) -> dict:
    """Gradients of sum(dout * out), with ``mean`` and ``rstd`` as the forward wrote them.
    Returns a dict of new tensors: dx (like x, contiguous), and fp32 dweight and dbias
    (None unless ``want_params``, by default where there is a weight)."""
    dev, dt, shape, lead, D, stride = _shape(x)
    dout_stride = _args.rows("dout", dout, x.dtype, shape, lead, D, dev)
    f32, row = torch.float32, shape[:-1]
    pw = _args.optional("weight", weight, f32, (D,), dev)
    pm, pr = _args.tensor("mean", mean, f32, row, dev), _args.tensor("rstd", rstd, f32, row, dev)
    if want_params is None:
        want_params = weight is not None
    dx, = _args.new(stream, x, shape)
    param = (D,) if want_params else None
    dw, db = _args.new(stream, mean, param, param)
    _args.done(_args.entry("kda_layer_norm_bwd")(
        dout.data_ptr(), dout_stride, x.data_ptr(), stride, pw, pm, pr, dx.data_ptr(),
        dw.data_ptr() if want_params else None, db.data_ptr() if want_params else None, dt, math.prod(row), D,
        _args.stream_handle(stream, dev)))
    return {"dx": dx, "dweight": dw, "dbias": db}

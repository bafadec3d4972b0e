"""RMS norm over the last axis with the residual's addition, forward and backward (C entry
points kda_rms_norm_fwd and kda_rms_norm_bwd of include/kda.h):

    h = x + residual (rounded to x's type),   out = h * rstd * weight,
    rstd = 1 / sqrt(mean(h^2) + eps)

``x`` and ``residual`` are [..., D] in bf16, fp16 or fp32, rows evenly spaced (a slice of a
wider tensor qualifies); ``weight`` is fp32 [D] or None; ``rstd`` is fp32.  The output is of
x's type, or in 8 bits with a scale for each block of 128 columns, as ``fp8.matmul`` reads it
(``fp8.empty`` makes such a pair).
"""
from __future__ import annotations

import math

import torch

from . import _args, fp8


def _shape(x):
    dt, shape = _args.dtype_code("x", x), x.shape
    lead = len(shape) - 1
    if lead < 0:
        raise ValueError("x must have at least one dimension")
    dev = _args.device("x", x)
    return dev, dt, shape, lead, shape[-1], shape[0] if lead == 1 else math.prod(shape[:-1]), \
        *_args.matrix("x", x, x.dtype, shape, lead, dev)


def _maybe(name, t, x, shape, lead, dev):
    """Data pointer and row stride of an optional tensor like ``x``."""
    return (None, 0) if t is None else _args.matrix(name, t, x.dtype, shape, lead, dev)


def _plain_fwd(x, weight, eps, out, residual, residual_out, rstd, scales) -> bool:
    """The forward pass of matrices on the current stream, like fp8's _plain_ functions: the same
    checks, each attribute looked at once; False, and nothing done, where it is not that plain."""
    try:
        kind, (R, D), dev = x.dtype, x.shape, x.get_device()
        dt, ot = _args.DTYPES[kind], out.dtype
        if out.shape != (R, D) or not 0 <= dev == out.get_device() == _args.current_device():
            return False
        wx, wo, ps, ws, pr, wr, po, wro = _args.width(x, D), _args.width(out, D), None, 0, None, 0, None, 0
        if ot is kind:
            code = dt
            if scales is not None:
                return False
        else:
            code, n = fp8.DTYPES[ot], -(-D // 128)
            if scales.shape != (R, n) or scales.dtype is not fp8.SCALE or scales.get_device() != dev:
                return False
            ps, ws = scales.data_ptr(), _args.width(scales, n)
        if residual is not None:
            if residual.dtype is not kind or residual.shape != (R, D) or residual.get_device() != dev:
                return False
            pr, wr = residual.data_ptr(), _args.width(residual, D)
        if residual_out is not None:
            if residual is None or residual_out.dtype is not kind or residual_out.shape != (R, D) or residual_out.get_device() != dev:
                return False
            po, wro = residual_out.data_ptr(), _args.width(residual_out, D)
    except (AttributeError, KeyError, TypeError, ValueError):
        return False
    if wx < 0 or wo < 0 or ws < 0 or wr < 0 or wro < 0:
        return False
    f32 = torch.float32
    _args.done(_args.entry("kda_rms_norm_fwd")(
        x.data_ptr(), wx, pr, wr, _args.optional("weight", weight, f32, (D,), dev), eps, out.data_ptr(), wo, code, ps, ws, po, wro,
        _args.optional("rstd", rstd, f32, (R,), dev), dt, R, D, _args.stream_handle(None, dev)))
    return True


def rms_norm_fwd(x, weight, eps, out, residual=None, residual_out=None, rstd=None, scales=None, stream=None) -> None:
    """Writes ``out`` [..., D] and, where given, ``residual_out`` (the sum h, like ``x``) and
    ``rstd`` (fp32, one value per row), asynchronously on ``stream`` (default: the current torch
    stream).  ``out`` is of x's type (it may be ``x`` or ``residual``), or torch.float8_e4m3fn
    or torch.float8_e5m2 with ``scales`` [..., ceil(D/128)] of torch.float8_e8m0fnu;
    ``residual_out`` may be ``x`` or ``residual``."""
    if stream is None and _plain_fwd(x, weight, eps, out, residual, residual_out, rstd, scales):
        return
    dev, dt, shape, lead, D, rows, px, xs = _shape(x)
    code, row = fp8.DTYPES.get(out.dtype) if isinstance(out, torch.Tensor) else None, shape[:-1]
    if code is None:
        if scales is not None:
            raise ValueError("scales belong to an 8-bit out")
        code, ps, ss = dt, None, 0
        pout, os = _args.matrix("out", out, x.dtype, shape, lead, dev)
    else:
        if scales is None:
            raise ValueError("an 8-bit out needs scales")
        pout, os = _args.matrix("out", out, out.dtype, shape, lead, dev)
        ps, ss = _args.matrix("scales", scales, fp8.SCALE, (*row, fp8.blocks(D)), lead, dev)
    if residual_out is not None and residual is None:
        raise ValueError("residual_out needs a residual")
    pr, rs = _maybe("residual", residual, x, shape, lead, dev)
    po, ros = _maybe("residual_out", residual_out, x, shape, lead, dev)
    f32 = torch.float32
    _args.done(_args.entry("kda_rms_norm_fwd")(
        px, xs, pr, rs, _args.optional("weight", weight, f32, (D,), dev), eps, pout, os, code, ps, ss, po, ros,
        _args.optional("rstd", rstd, f32, row, dev), dt, rows, D, _args.stream_handle(stream, dev)))


def _plain_bwd(dout, x, weight, rstd, dresidual, want_dweight):
    """The backward pass, likewise: its result, or None."""
    try:
        kind, (R, D), dev = x.dtype, x.shape, x.get_device()
        dt, wx, wd, pr, wr = _args.DTYPES[kind], _args.width(x, D), _args.width(dout, D), None, 0
        if dout.dtype is not kind or dout.shape != (R, D) or not 0 <= dev == dout.get_device() == _args.current_device():
            return None
        if dresidual is not None:
            if dresidual.dtype is not kind or dresidual.shape != (R, D) or dresidual.get_device() != dev:
                return None
            pr, wr = dresidual.data_ptr(), _args.width(dresidual, D)
    except (AttributeError, KeyError, TypeError, ValueError):
        return None
    if wx < 0 or wd < 0 or wr < 0:
        return None
    f32 = torch.float32
    pw, ps = _args.optional("weight", weight, f32, (D,), dev), _args.tensor("rstd", rstd, f32, (R,), dev)
    dx, dw = torch.empty_like(x, memory_format=torch.contiguous_format), None
    if weight is not None if want_dweight is None else want_dweight:
        dw = rstd.new_empty((D,)) if weight is None else torch.empty_like(weight)
    _args.done(_args.entry("kda_rms_norm_bwd")(dout.data_ptr(), wd, x.data_ptr(), wx, pw, ps, pr, wr, dx.data_ptr(),
                                               None if dw is None else dw.data_ptr(), dt, R, D, _args.stream_handle(None, dev)))
    return {"dx": dx, "dweight": dw}


def rms_norm_bwd(dout, x, weight, rstd, dresidual=None, want_dweight=None, stream=None) -> dict:
    """Gradients of sum(dout * out) + sum(dresidual * residual_out); ``x`` is the sum h that was
    normed and ``rstd`` what the forward wrote.  Returns a dict of new tensors: dx (like x,
    contiguous: the gradient of the forward's x and of its residual) and fp32 dweight (None
    unless ``want_dweight``, by default where there is a weight)."""
    if stream is None and (plain := _plain_bwd(dout, x, weight, rstd, dresidual, want_dweight)):
        return plain
    dev, dt, shape, lead, D, rows, px, xs = _shape(x)
    pdo, dos = _args.matrix("dout", dout, x.dtype, shape, lead, dev)
    pd, ds = _maybe("dresidual", dresidual, x, shape, lead, dev)
    f32 = torch.float32
    pw, pr = _args.optional("weight", weight, f32, (D,), dev), _args.tensor("rstd", rstd, f32, shape[:-1], dev)
    if want_dweight is None:
        want_dweight = weight is not None
    dx, = _args.new(stream, x, shape)
    dw, = _args.new(stream, rstd, (D,) if want_dweight else None)
    _args.done(_args.entry("kda_rms_norm_bwd")(
        pdo, dos, px, xs, pw, pr, pd, ds, dx.data_ptr(), None if dw is None else dw.data_ptr(), dt, rows, D,
        _args.stream_handle(stream, dev)))
    return {"dx": dx, "dweight": dw}

"""Causal depthwise short convolution with its activation, forward and backward (C entry
points kda_short_conv_fwd and kda_short_conv_bwd of include/kda.h):

    y_t[c] = bias[c] + sum_j weight[c, j] * x_{t-(W-1)+j}[c],   out = y * sigmoid(y)

over 2 to 4 taps.  ``x`` is [B, T, D] in bf16, fp16 or fp32, tokens evenly spaced (a slice
of a wider projection qualifies); ``weight`` fp32 [D, W], ``bias`` fp32 [D] or None.  The
state of a sequence, [W-1, D] of x's type, is its last W-1 input rows, oldest first.
"""
from __future__ import annotations

import torch

from . import _args

ACTIVATIONS = {None: 0, "silu": 1}   # kda_activation


def _check(x, weight, bias, activation):
    dt, shape = _args.dtype_code("x", x), x.shape
    if len(shape) != 3:
        raise ValueError("x must be [B, T, D]")
    D, f32 = shape[2], torch.float32
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D, W] tensor")
    W = weight.shape[1]
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    dev = _args.device("x", x)
    return (dev, dt, shape, W, _args.rows("x", x, x.dtype, shape, 2, D, dev), act,
            _args.tensor("weight", weight, f32, (D, W), dev), _args.optional("bias", bias, f32, (D,), dev))


def short_conv_fwd(x, weight, bias, out, activation="silu", initial_state=None, final_state=None,
                   cu_seqlens=None, stream=None) -> None:
    """Writes ``out`` (like ``x``) and, where given, ``final_state`` [N, W-1, D] (which may
    be ``initial_state`` itself) in place, asynchronously on ``stream`` (default: the
    current torch stream)."""
    dev, dt, shape, W, stride, act, pw, pb = _check(x, weight, bias, activation)
    B, T, D = shape
    out_stride = _args.rows("out", out, x.dtype, shape, 2, D, dev)
    num_seqs, cu = _args.sequences(cu_seqlens, dev)
    state = (num_seqs or B, W - 1, D)
    _args.done(_args.entry("kda_short_conv_fwd")(
        x.data_ptr(), stride, pw, pb, act, out.data_ptr(), out_stride, dt,
        _args.optional("initial_state", initial_state, x.dtype, state, dev),
        _args.optional("final_state", final_state, x.dtype, state, dev), cu, num_seqs, B, T, D, W,
        _args.stream_handle(stream, dev)))


def short_conv_bwd(x, weight, bias, dout, activation="silu", initial_state=None, dfinal=None,
                   cu_seqlens=None, want_dinit=True, stream=None) -> dict:
    """Gradients of L = sum(dout * out) + sum(dfinal * final_state); ``dfinal`` fp32
    [N, W-1, D] or None.  Returns a dict of new tensors: dx (x's type, contiguous), and fp32
    dweight, dbias (None without a bias) and dinit (None unless ``want_dinit``)."""
    dev, dt, shape, W, stride, act, pw, pb = _check(x, weight, bias, activation)
    B, T, D = shape
    dout_stride = _args.rows("dout", dout, x.dtype, shape, 2, D, dev)
    num_seqs, cu = _args.sequences(cu_seqlens, dev)
    state, f32 = (num_seqs or B, W - 1, D), torch.float32
    init = _args.optional("initial_state", initial_state, x.dtype, state, dev)
    dfin = _args.optional("dfinal", dfinal, f32, state, dev)
    dx, = _args.new(stream, x, shape)
    dw, db, dinit = _args.new(stream, weight, (D, W), None if bias is None else (D,), state if want_dinit else None)
    _args.done(_args.entry("kda_short_conv_bwd")(
        x.data_ptr(), stride, pw, pb, act, dt, init, dout.data_ptr(), dout_stride, dfin, cu, num_seqs, B, T, D, W,
        dx.data_ptr(), dw.data_ptr(), None if db is None else db.data_ptr(), None if dinit is None else dinit.data_ptr(),
        _args.stream_handle(stream, dev)))
    return {"dx": dx, "dweight": dw, "dbias": db, "dinit": dinit}

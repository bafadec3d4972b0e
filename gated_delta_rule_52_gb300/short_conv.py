"""Causal depthwise short convolution with its activation, forward and backward (C entry
points kda_short_conv_fwd and kda_short_conv_bwd of include/kda.h):

    y_t[c] = bias[c] + sum_j weight[c, j] * x_{t-(W-1)+j}[c],   out = y * sigmoid(y)

over 2 to 4 taps.  ``x`` is [B, T, D] in bf16, fp16 or fp32, tokens evenly spaced (a slice
of a wider projection qualifies); ``weight`` fp32 [D, W], ``bias`` fp32 [D] or None.  The
state of a sequence, [W-1, D] of x's type, is its last W-1 input rows, oldest first.
"""
from __future__ import annotations

import torch

from . import _args, kda

ACTIVATIONS = {None: 0, "silu": 1}   # kda_activation


def _check(x, weight, bias, activation, cu_seqlens):
    dt = _args.dtype_code("x", x)
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a [D, W] tensor")
    W = weight.shape[1]
    _args.check("weight", weight, torch.float32, (D, W))
    if bias is not None:
        _args.check("bias", bias, torch.float32, (D,))
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    return dt, (B, T, D, W), _args.rows("x", x, x.dtype, x.shape, 2), ACTIVATIONS[activation], \
        _args.sequences(cu_seqlens)


def short_conv_fwd(x, weight, bias, out, activation="silu", initial_state=None, final_state=None,
                   cu_seqlens=None, stream=None) -> None:
    """Writes ``out`` (like ``x``) and, where given, ``final_state`` [N, W-1, D] (which may
    be ``initial_state`` itself) in place, asynchronously on ``stream`` (default: the
    current torch stream)."""
    dt, (B, T, D, W), stride, act, num_seqs = _check(x, weight, bias, activation, cu_seqlens)
    out_stride = _args.rows("out", out, x.dtype, x.shape, 2)
    for name, s in (("initial_state", initial_state), ("final_state", final_state)):
        if s is not None:
            _args.check(name, s, x.dtype, (num_seqs or B, W - 1, D))
    p = _args.ptr
    _args.done(kda.lib().kda_short_conv_fwd(p(x), stride, p(weight), p(bias), act, p(out), out_stride, dt,
                                            p(initial_state), p(final_state), p(cu_seqlens), num_seqs, B, T, D, W,
                                            _args.stream_handle(stream)))


def short_conv_bwd(x, weight, bias, dout, activation="silu", initial_state=None, dfinal=None,
                   cu_seqlens=None, want_dinit=True, stream=None) -> dict:
    """Gradients of L = sum(dout * out) + sum(dfinal * final_state); ``dfinal`` fp32
    [N, W-1, D] or None.  Returns a dict of new tensors: dx (x's type, contiguous), and fp32
    dweight, dbias (None without a bias) and dinit (None unless ``want_dinit``)."""
    dt, (B, T, D, W), stride, act, num_seqs = _check(x, weight, bias, activation, cu_seqlens)
    dout_stride = _args.rows("dout", dout, x.dtype, x.shape, 2)
    N = num_seqs or B
    if initial_state is not None:
        _args.check("initial_state", initial_state, x.dtype, (N, W - 1, D))
    if dfinal is not None:
        _args.check("dfinal", dfinal, torch.float32, (N, W - 1, D))
    with _args.on(stream):
        dev = x.device
        r = {"dx": torch.empty((B, T, D), dtype=x.dtype, device=dev),
             "dweight": torch.empty((D, W), dtype=torch.float32, device=dev),
             "dbias": None if bias is None else torch.empty((D,), dtype=torch.float32, device=dev),
             "dinit": torch.empty((N, W - 1, D), dtype=torch.float32, device=dev) if want_dinit else None}
    p = _args.ptr
    _args.done(kda.lib().kda_short_conv_bwd(p(x), stride, p(weight), p(bias), act, dt, p(initial_state), p(dout),
                                            dout_stride, p(dfinal), p(cu_seqlens), num_seqs, B, T, D, W, p(r["dx"]),
                                            p(r["dweight"]), p(r["dbias"]), p(r["dinit"]),
                                            _args.stream_handle(stream)))
    return r

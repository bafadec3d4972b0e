"""Gated linear recurrence, the delta rule's vector-state sibling (C entry points
kda_glr_fwd and kda_glr_bwd of include/kda.h).  Per channel, with the state in fp32:

    h_t = exp(gk_t) h_{t-1} + sigmoid(i_t) x_t,   out_t = h_t
    gk_t = lower_bound * sigmoid(exp(A_log) * (g_t + dt_bias))      (kda_fwd's gate), or
    gk_t = -exp(A_log) * softplus(g_t + dt_bias)                    (``lower_bound=None``)

Tensors are [B, T, H, K] in bf16, fp16 or fp32; any B, T, H, K, single tokens included.
Inputs may be slices of a wider tensor (one projection's output) as long as a token's
channels are contiguous and the tokens evenly spaced.
"""
from __future__ import annotations

import torch

from . import _args

# Packed rows from one checkpoint to the next (KDA_GLR_CHECKPOINT_ROWS).
CHECKPOINT_ROWS = 64


def checkpoint_shape(B: int, T: int, H: int, K: int) -> tuple:
    """Shape of the fp32 tensor of checkpoints of a [B, T, H, K] call."""
    return (-(-B * T // CHECKPOINT_ROWS), H, K)


def _check(x, i, g, A_log, dt_bias):
    dt = _args.dtype_code("x", x)
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, K]")
    shape = x.shape
    B, T, H, K = shape
    D, dtype, rows, dev = H * K, x.dtype, _args.rows, _args.device("x", x)
    f32 = torch.float32
    return (dev, dt, shape, D, rows("x", x, dtype, shape, 2, D, dev), rows("i", i, dtype, shape, 2, D, dev),
            rows("g", g, dtype, shape, 2, D, dev), _args.tensor("A_log", A_log, f32, (H,), dev),
            _args.tensor("dt_bias", dt_bias, f32, (H, K), dev))


def glr_fwd(x, i, g, out, A_log, dt_bias, lower_bound, initial_state=None, final_state=None,
            cu_seqlens=None, checkpoints=None, stream=None) -> None:
    """Writes ``out`` [B,T,H,K] (and ``final_state`` [N,H,K], bf16 or fp32, which may be
    ``initial_state`` itself) in place, asynchronously on ``stream`` (default: the current
    torch stream).  ``checkpoints`` (fp32, ``checkpoint_shape``) takes the states that
    ``glr_bwd`` starts from."""
    dev, dt, shape, D, xs, is_, gs, pA, pt = _check(x, i, g, A_log, dt_bias)
    B, T, H, K = shape
    out_stride = _args.rows("out", out, x.dtype, shape, 2, D, dev)
    num_seqs, cu = _args.sequences(cu_seqlens, dev)
    code, init, fin = _args.states(initial_state, final_state, (num_seqs or B, H, K), dev)
    ck = None if checkpoints is None else _args.tensor("checkpoints", checkpoints, torch.float32, checkpoint_shape(B, T, H, K), dev)
    _args.done(_args.entry("kda_glr_fwd")(
        x.data_ptr(), i.data_ptr(), g.data_ptr(), xs, is_, gs, out.data_ptr(), out_stride, dt, pA, pt, lower_bound or 0.0,
        lower_bound is None, init, fin, code, cu, num_seqs, B, T, H, K, ck, _args.stream_handle(stream, dev)))


def glr_bwd(x, i, g, A_log, dt_bias, lower_bound, dout, initial_state=None, dfinal=None,
            cu_seqlens=None, checkpoints=None, want_dinit=True, stream=None) -> dict:
    """Gradients of L = sum(dout * out) + sum(dfinal * final_state).  ``dout`` like ``x``;
    ``dfinal`` fp32 [N,H,K] or None; ``checkpoints`` as ``glr_fwd`` left them for these
    inputs, or None (the states are recomputed).  Returns a dict of new tensors: dx, di, dg
    in the inputs' type, and fp32 dA_log, ddt_bias and dinit (None unless ``want_dinit``)."""
    dev, dt, shape, D, xs, is_, gs, pA, pt = _check(x, i, g, A_log, dt_bias)
    B, T, H, K = shape
    ds = _args.rows("dout", dout, x.dtype, shape, 2, D, dev)
    num_seqs, cu = _args.sequences(cu_seqlens, dev)
    state, f32 = (num_seqs or B, H, K), torch.float32
    code, init, _ = _args.states(initial_state, None, state, dev)
    dfin = _args.optional("dfinal", dfinal, f32, state, dev)
    ck = None if checkpoints is None else _args.tensor("checkpoints", checkpoints, f32, checkpoint_shape(B, T, H, K), dev)
    dx, di, dg = _args.new(stream, x, shape, shape, shape)
    dA_log, ddt_bias, dinit = _args.new(stream, A_log, (H,), (H, K), state if want_dinit else None)
    _args.done(_args.entry("kda_glr_bwd")(
        x.data_ptr(), i.data_ptr(), g.data_ptr(), xs, is_, gs, dt, pA, pt, lower_bound or 0.0, lower_bound is None, init,
        code, ck, dout.data_ptr(), ds, dfin, cu, num_seqs, B, T, H, K, dx.data_ptr(), di.data_ptr(), dg.data_ptr(),
        dA_log.data_ptr(), ddt_bias.data_ptr(), None if dinit is None else dinit.data_ptr(),
        _args.stream_handle(stream, dev)))
    return {"dx": dx, "di": di, "dg": dg, "dA_log": dA_log, "ddt_bias": ddt_bias, "dinit": dinit}

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

from . import _args, kda

# Packed rows from one checkpoint to the next (KDA_GLR_CHECKPOINT_ROWS).
CHECKPOINT_ROWS = 64


def checkpoint_shape(B: int, T: int, H: int, K: int) -> tuple:
    """Shape of the fp32 tensor of checkpoints of a [B, T, H, K] call."""
    return (-(-B * T // CHECKPOINT_ROWS), H, K)


def _check(x, i, g, A_log, dt_bias, cu_seqlens):
    dt = _args.dtype_code("x", x)
    if x.dim() != 4:
        raise ValueError("x must be [B, T, H, K]")
    B, T, H, K = shape = x.shape
    strides = [_args.rows(n, t, x.dtype, shape, 2) for n, t in (("x", x), ("i", i), ("g", g))]
    _args.check("A_log", A_log, torch.float32, (H,))
    _args.check("dt_bias", dt_bias, torch.float32, (H, K))
    return dt, shape, strides, _args.sequences(cu_seqlens)


def glr_fwd(x, i, g, out, A_log, dt_bias, lower_bound, initial_state=None, final_state=None,
            cu_seqlens=None, checkpoints=None, stream=None) -> None:
    """Writes ``out`` [B,T,H,K] (and ``final_state`` [N,H,K], bf16 or fp32, which may be
    ``initial_state`` itself) in place, asynchronously on ``stream`` (default: the current
    torch stream).  ``checkpoints`` (fp32, ``checkpoint_shape``) takes the states that
    ``glr_bwd`` starts from."""
    dt, (B, T, H, K), strides, num_seqs = _check(x, i, g, A_log, dt_bias, cu_seqlens)
    out_stride = _args.rows("out", out, x.dtype, x.shape, 2)
    N = num_seqs or B
    code = kda.state_dtype_code(initial_state, final_state)
    for name, s in (("initial_state", initial_state), ("final_state", final_state)):
        if s is not None:
            _args.check(name, s, s.dtype, (N, H, K))
    if checkpoints is not None:
        _args.check("checkpoints", checkpoints, torch.float32, checkpoint_shape(B, T, H, K))
    p = _args.ptr
    _args.done(kda.lib().kda_glr_fwd(
        p(x), p(i), p(g), *strides, p(out), out_stride, dt, p(A_log), p(dt_bias), lower_bound or 0.0,
        lower_bound is None, p(initial_state), p(final_state), code, p(cu_seqlens), num_seqs, B, T, H, K,
        p(checkpoints), _args.stream_handle(stream)))


def glr_bwd(x, i, g, A_log, dt_bias, lower_bound, dout, initial_state=None, dfinal=None,
            cu_seqlens=None, checkpoints=None, want_dinit=True, stream=None) -> dict:
    """Gradients of L = sum(dout * out) + sum(dfinal * final_state).  ``dout`` like ``x``;
    ``dfinal`` fp32 [N,H,K] or None; ``checkpoints`` as ``glr_fwd`` left them for these
    inputs, or None (the states are recomputed).  Returns a dict of new tensors: dx, di, dg
    in the inputs' type, and fp32 dA_log, ddt_bias and dinit (None unless ``want_dinit``)."""
    dt, (B, T, H, K), strides, num_seqs = _check(x, i, g, A_log, dt_bias, cu_seqlens)
    dout_stride = _args.rows("dout", dout, x.dtype, x.shape, 2)
    N = num_seqs or B
    code = kda.state_dtype_code(initial_state, None)
    if initial_state is not None:
        _args.check("initial_state", initial_state, initial_state.dtype, (N, H, K))
    if dfinal is not None:
        _args.check("dfinal", dfinal, torch.float32, (N, H, K))
    if checkpoints is not None:
        _args.check("checkpoints", checkpoints, torch.float32, checkpoint_shape(B, T, H, K))
    with _args.on(stream):
        dev = x.device
        r = {k: torch.empty((B, T, H, K), dtype=x.dtype, device=dev) for k in ("dx", "di", "dg")}
        r["dA_log"] = torch.empty((H,), dtype=torch.float32, device=dev)
        r["ddt_bias"] = torch.empty((H, K), dtype=torch.float32, device=dev)
        r["dinit"] = torch.empty((N, H, K), dtype=torch.float32, device=dev) if want_dinit else None
    p = _args.ptr
    _args.done(kda.lib().kda_glr_bwd(
        p(x), p(i), p(g), *strides, dt, p(A_log), p(dt_bias), lower_bound or 0.0, lower_bound is None,
        p(initial_state), code, p(checkpoints), p(dout), dout_stride, p(dfinal), p(cu_seqlens), num_seqs,
        B, T, H, K, p(r["dx"]), p(r["di"]), p(r["dg"]), p(r["dA_log"]), p(r["ddt_bias"]), p(r["dinit"]),
        _args.stream_handle(stream)))
    return r

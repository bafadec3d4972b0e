"""Tensors in 8-bit floating point with a power-of-two scale for each block of 128, and their
product (C entry points kda_fp8_quantize, kda_fp8_dequantize and kda_fp8_matmul of
include/kda.h):

    q = x / scale,   out[m, n] = add[m, n] + sum_k (a[m, k] a_scale) (b[n, k] b_scale)

Elements are torch.float8_e4m3fn or torch.float8_e5m2, scales torch.float8_e8m0fnu.  A scale
belongs to 128 neighbours of a row, [rows, ceil(cols/128)], or (``tile``, for weights) to a tile
of 128 rows by 128 columns, [ceil(rows/128), ceil(cols/128)].  The tensor cores multiply the
scales in, so the product costs what one without scales does.

A projection y = x W^T and its gradients, in tokens x of [M, K] and weights W of [N, K]:

    q, s = fp8.empty(M, K);  fp8.quantize(x, q, s)           # or rms_norm.rms_norm_fwd's output
    fp8.matmul(q, s, wq, ws, y)                              # W by tiles: wq, ws, and wt, wts = W^T
    fp8.quantize(dy, dq, ds, qt=dqt, scales_t=dst)           # both ways in one pass
    fp8.matmul(dq, ds, wt, wts, dx)                          # dx = dy W
    fp8.matmul(dqt, dst, xt, xts, dW, add=dW)                # dW += dy^T x
"""
from __future__ import annotations

import math

import torch

from . import _args

DTYPES = {torch.float8_e4m3fn: 4, torch.float8_e5m2: 5}   # kda_dtype
SCALE = torch.float8_e8m0fnu
BLOCK = 128                                               # KDA_FP8_BLOCK


def blocks(n: int) -> int:
    """Blocks of 128 in a row of n elements."""
    return -(-n // BLOCK)


def empty(rows: int, cols: int, dtype=torch.float8_e4m3fn, tile: bool = False, device="cuda") -> tuple:
    """New (q, scales) of a [rows, cols] tensor, uninitialised, with rows as ``matmul`` reads
    them: 16 bytes aligned, those of the scales 4."""
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be float8_e4m3fn or float8_e5m2, got {dtype}")
    lines, n = blocks(rows) if tile else rows, blocks(cols)
    return (torch.empty(rows, -(-cols // 16) * 16, dtype=dtype, device=device)[:, :cols],
            torch.empty(lines, -(-n // 4) * 4, dtype=SCALE, device=device)[:, :n])


def _code(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float8_e4m3fn or float8_e5m2, got {t.dtype}")
    return code


def _scales(name, s, shape, lead, tile, dev):
    """Pointer and row stride of the scales of an 8-bit tensor of this shape."""
    n = -(-shape[-1] // BLOCK)
    if tile:
        return _args.matrix(name, s, SCALE, (-(-math.prod(shape[:-1]) // BLOCK), n), 1, dev)
    return _args.matrix(name, s, SCALE, (shape[0], n) if lead == 1 else (*shape[:-1], n), lead, dev)


def _tiled(name, s, shape, lead):
    """Whether the scales of an 8-bit tensor of this shape are those of tiles."""
    if not isinstance(s, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return s.dim() != lead + 1 or s.shape[0] != shape[0]


def _pair(name, q, s, code, shape, tile, dev):
    """Pointers and row strides of an 8-bit tensor that is written, and of its scales."""
    if q is None:
        if s is not None:
            raise ValueError(f"scales without {name}")
        return None, 0, None, 0
    if s is None:
        raise ValueError(f"{name} without its scales")
    if _code(name, q) != code:
        raise ValueError("q and qt must be of one type")
    lead = len(shape) - 1
    return *_args.matrix(name, q, q.dtype, shape, lead, dev), *_scales(f"scales of {name}", s, shape, lead, tile, dev)


def quantize(x, q=None, scales=None, qt=None, scales_t=None, tile=False, stream=None) -> None:
    """Writes ``x`` [..., cols] (bf16, fp16 or fp32, rows evenly spaced) in 8 bits to ``q``, shaped
    like x, and ``scales``, and its transpose to ``qt`` [cols, rows] and ``scales_t``, whose blocks
    lie along x's columns; one pass over x does both.  Asynchronous on ``stream`` (default: the
    current torch stream)."""
    dt, shape = _args.dtype_code("x", x), x.shape
    lead = len(shape) - 1
    if lead < 1:
        raise ValueError("x must have at least two dimensions")
    if q is None and qt is None:
        raise ValueError("q or qt must be given")
    cols, dev = shape[-1], _args.device("x", x)
    rows = shape[0] if lead == 1 else math.prod(shape[:-1])
    px, xs = _args.matrix("x", x, x.dtype, shape, lead, dev)
    code = _code("q" if q is not None else "qt", q if q is not None else qt)
    pq, qs, ps, ss = _pair("q", q, scales, code, shape, tile, dev)
    pt, ts, pst, sts = _pair("qt", qt, scales_t, code, (cols, rows), tile, dev)
    _args.done(_args.entry("kda_fp8_quantize")(px, xs, dt, pq, qs, ps, ss, pt, ts, pst, sts, code, bool(tile), rows, cols,
                                               _args.stream_handle(stream, dev)))


def dequantize(q, scales, out, stream=None) -> None:
    """Writes the values that ``q`` [..., cols] with ``scales`` (of rows, or of tiles) stands for
    to ``out`` (bf16, fp16 or fp32, shaped like q)."""
    code, shape = _code("q", q), q.shape
    lead = len(shape) - 1
    if lead < 1:
        raise ValueError("q must have at least two dimensions")
    dev, dt, tile = _args.device("q", q), _args.dtype_code("out", out), _tiled("scales", scales, shape, lead)
    pq, qs = _args.matrix("q", q, q.dtype, shape, lead, dev)
    ps, ss = _scales("scales", scales, shape, lead, tile, dev)
    po, os = _args.matrix("out", out, out.dtype, shape, lead, dev)
    _args.done(_args.entry("kda_fp8_dequantize")(pq, qs, code, ps, ss, tile, po, os, dt, shape[0] if lead == 1 else math.prod(shape[:-1]),
                                                 shape[-1], _args.stream_handle(stream, dev)))


def matmul(a, a_scales, b, b_scales, out, add=None, stream=None) -> None:
    """Writes out[..., n] = add[..., n] + sum_k a[..., k] b[n, k], of the values that the 8-bit
    tensors ``a`` [..., K] and ``b`` [N, K] stand for, asynchronously on ``stream`` (default: the
    current torch stream).  Scales are those of rows or of tiles, by their shape.  ``out``
    [..., N] is bf16, fp16 or fp32, ``add`` None or like it (it may be ``out``, or one row
    expanded to all, a bias).  Rows of a and b
    start at multiples of 16 bytes, those of the scales at multiples of 4, as ``empty`` lays them
    out; sums are fp32."""
    ca, cb, dt, sa, sb = _code("a", a), _code("b", b), _args.dtype_code("out", out), a.shape, b.shape
    lead = len(sa) - 1
    if lead < 1 or len(sb) != 2:
        raise ValueError("a must be [..., K] and b [N, K]")
    K, N, dev = sa[-1], sb[0], _args.device("a", a)
    M, shape = (sa[0], (sa[0], N)) if lead == 1 else (math.prod(sa[:-1]), (*sa[:-1], N))
    ta, tb = _tiled("a_scales", a_scales, sa, lead), _tiled("b_scales", b_scales, sb, 1)
    pa, as_ = _args.matrix("a", a, a.dtype, sa, lead, dev)
    psa, sas = _scales("a_scales", a_scales, sa, lead, ta, dev)
    pb, bs = _args.matrix("b", b, b.dtype, (N, K), 1, dev)
    psb, sbs = _scales("b_scales", b_scales, sb, 1, tb, dev)
    po, os = _args.matrix("out", out, out.dtype, shape, lead, dev)
    pp, ps = (None, 0) if add is None else _args.matrix("add", add, out.dtype, shape, lead, dev)
    _args.done(_args.entry("kda_fp8_matmul")(pa, as_, ca, psa, sas, ta, pb, bs, cb, psb, sbs, tb, po, os, pp, ps, dt, M, N, K,
                                             _args.stream_handle(stream, dev)))

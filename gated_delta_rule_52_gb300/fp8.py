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


def _scale_rows(name, s, shape, tile, dev):
    """Row stride of the scales of an 8-bit tensor of this shape."""
    n = blocks(shape[-1])
    if tile:
        return _args.rows(name, s, SCALE, (blocks(math.prod(shape[:-1])), n), 1, n, dev)
    return _args.rows(name, s, SCALE, (*shape[:-1], n), len(shape) - 1, n, dev)


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
    return (q.data_ptr(), _args.rows(name, q, q.dtype, shape, lead, shape[-1], dev), s.data_ptr(),
            _scale_rows(f"scales of {name}", s, shape, tile, dev))


def quantize(x, q=None, scales=None, qt=None, scales_t=None, tile=False, stream=None) -> None:
    """Writes ``x`` [..., cols] (bf16, fp16 or fp32, rows evenly spaced) in 8 bits to ``q``, shaped
    like x, and ``scales``, and its transpose to ``qt`` [cols, rows] and ``scales_t``, whose blocks
    lie along x's columns; one pass over x does both.  Asynchronous on ``stream`` (default: the
    current torch stream)."""
    dt, shape = _args.dtype_code("x", x), x.shape
    if len(shape) < 2:
        raise ValueError("x must have at least two dimensions")
    if q is None and qt is None:
        raise ValueError("q or qt must be given")
    cols, lead, dev = shape[-1], len(shape) - 1, _args.device("x", x)
    stride, rows = _args.rows("x", x, x.dtype, shape, lead, cols, dev), math.prod(shape[:-1])
    code = _code("q" if q is not None else "qt", q if q is not None else qt)
    pq, qs, ps, ss = _pair("q", q, scales, code, shape, tile, dev)
    pt, ts, pst, sts = _pair("qt", qt, scales_t, code, (cols, rows), tile, dev)
    _args.done(_args.entry("kda_fp8_quantize")(x.data_ptr(), stride, dt, pq, qs, ps, ss, pt, ts, pst, sts, code, bool(tile), rows,
                                               cols, _args.stream_handle(stream, dev)))


def _tiled(name, s, shape):
    """Whether the scales of an 8-bit tensor of this shape are those of tiles."""
    if not isinstance(s, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return s.shape != (*shape[:-1], blocks(shape[-1]))


def dequantize(q, scales, out, stream=None) -> None:
    """Writes the values that ``q`` [..., cols] with ``scales`` (of rows, or of tiles) stands for
    to ``out`` (bf16, fp16 or fp32, shaped like q)."""
    code, shape = _code("q", q), q.shape
    if len(shape) < 2:
        raise ValueError("q must have at least two dimensions")
    cols, lead, dev = shape[-1], len(shape) - 1, _args.device("q", q)
    dt, tile = _args.dtype_code("out", out), _tiled("scales", scales, shape)
    _args.done(_args.entry("kda_fp8_dequantize")(
        q.data_ptr(), _args.rows("q", q, q.dtype, shape, lead, cols, dev), code, scales.data_ptr(),
        _scale_rows("scales", scales, shape, tile, dev), tile, out.data_ptr(),
        _args.rows("out", out, out.dtype, shape, lead, cols, dev), dt, math.prod(shape[:-1]), cols, _args.stream_handle(stream, dev)))


def matmul(a, a_scales, b, b_scales, out, add=None, stream=None) -> None:
    """Writes out[..., n] = add[..., n] + sum_k a[..., k] b[n, k], of the values that the 8-bit
    tensors ``a`` [..., K] and ``b`` [N, K] stand for, asynchronously on ``stream`` (default: the
    current torch stream).  Scales are those of rows or of tiles, by their shape.  ``out``
    [..., N] is bf16, fp16 or fp32, ``add`` None or like it (it may be ``out``).  Rows of a and b
    start at multiples of 16 bytes, those of the scales at multiples of 4, as ``empty`` lays them
    out; sums are fp32."""
    ca, cb, sa, sb = _code("a", a), _code("b", b), a.shape, b.shape
    if len(sa) < 2 or len(sb) != 2:
        raise ValueError("a must be [..., K] and b [N, K]")
    K, N, lead, dev = sa[-1], sb[0], len(sa) - 1, _args.device("a", a)
    dt, shape = _args.dtype_code("out", out), (*sa[:-1], N)
    ta, tb = _tiled("a_scales", a_scales, sa), _tiled("b_scales", b_scales, sb)
    rows = _args.rows
    _args.done(_args.entry("kda_fp8_matmul")(
        a.data_ptr(), rows("a", a, a.dtype, sa, lead, K, dev), ca, a_scales.data_ptr(),
        _scale_rows("a_scales", a_scales, sa, ta, dev), ta,
        b.data_ptr(), rows("b", b, b.dtype, (N, K), 1, K, dev), cb, b_scales.data_ptr(),
        _scale_rows("b_scales", b_scales, sb, tb, dev), tb,
        out.data_ptr(), rows("out", out, out.dtype, shape, lead, N, dev),
        None if add is None else add.data_ptr(), 0 if add is None else rows("add", add, out.dtype, shape, lead, N, dev), dt,
        math.prod(sa[:-1]), N, K, _args.stream_handle(stream, dev)))

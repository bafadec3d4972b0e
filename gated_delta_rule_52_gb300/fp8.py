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


# A short call's time is that of its checks.  The functions with _plain_ in front take matrices on the
# current stream and look once at each attribute; they make the same checks as the function itself
# and do nothing and return False where anything is not as it should be, or not this plain: the
# function then says what.  (A product's call: 7.5 us instead of 10.3.)


def _plain_quantize(x, q, scales, qt, scales_t, tile) -> bool:
    try:
        dt, (R, C), dev = _args.DTYPES[x.dtype], x.shape, x.get_device()
        wx, br, bc = _args.width(x, C), -(-R // BLOCK), -(-C // BLOCK)
        if not 0 <= dev == _args.current_device() or wx < 0:
            return False
        code = pq = ps = pt = pst = None
        wq = ws = wt = wst = 0
        if q is not None:
            code = DTYPES[q.dtype]
            if q.shape != (R, C) or scales.shape != (br if tile else R, bc) or scales.dtype is not SCALE or not q.get_device() == scales.get_device() == dev:
                return False
            pq, wq, ps, ws = q.data_ptr(), _args.width(q, C), scales.data_ptr(), _args.width(scales, bc)
        elif scales is not None:
            return False
        if qt is not None:
            ct = DTYPES[qt.dtype]
            if (code is not None and ct != code) or qt.shape != (C, R) or scales_t.shape != (bc if tile else C, br) or \
                    scales_t.dtype is not SCALE or not qt.get_device() == scales_t.get_device() == dev:
                return False
            code, pt, wt, pst, wst = ct, qt.data_ptr(), _args.width(qt, R), scales_t.data_ptr(), _args.width(scales_t, br)
        elif scales_t is not None or code is None:
            return False
    except (AttributeError, KeyError, TypeError, ValueError):
        return False
    if wq < 0 or ws < 0 or wt < 0 or wst < 0:
        return False
    _args.done(_args.entry("kda_fp8_quantize")(x.data_ptr(), wx, dt, pq, wq, ps, ws, pt, wt, pst, wst, code, bool(tile), R, C,
                                               _args.stream_handle(None, dev)))
    return True


def _plain_dequantize(q, scales, out) -> bool:
    try:
        code, dt, (R, C), (Ro, Co), (Rs, Cs), dev = DTYPES[q.dtype], _args.DTYPES[out.dtype], q.shape, out.shape, scales.shape, q.get_device()
    except (AttributeError, KeyError, TypeError, ValueError):
        return False
    tile, n = Rs != R, -(-C // BLOCK)
    if R != Ro or C != Co or Cs != n or (tile and Rs != -(-R // BLOCK)) or scales.dtype is not SCALE or \
            not 0 <= dev == out.get_device() == scales.get_device() == _args.current_device():
        return False
    wq, ws, wo = _args.width(q, C), _args.width(scales, n), _args.width(out, C)
    if wq < 0 or ws < 0 or wo < 0:
        return False
    _args.done(_args.entry("kda_fp8_dequantize")(q.data_ptr(), wq, code, scales.data_ptr(), ws, tile, out.data_ptr(), wo, dt, R, C,
                                                 _args.stream_handle(None, dev)))
    return True


def _plain_matmul(a, a_scales, b, b_scales, out, add) -> bool:
    try:
        ca, cb, dt = DTYPES[a.dtype], DTYPES[b.dtype], _args.DTYPES[out.dtype]
        (M, K), (N, L), (Mo, No), (Ma, Ka), (Nb, Kb) = a.shape, b.shape, out.shape, a_scales.shape, b_scales.shape
        dev, n = a.get_device(), -(-K // BLOCK)
        pp, wp = None, 0
        if add is not None:
            if add.dtype is not out.dtype or add.shape != (M, N) or add.get_device() != dev:
                return False
            pp, wp = add.data_ptr(), _args.width(add, N)
    except (AttributeError, KeyError, TypeError, ValueError):
        return False
    ta, tb = Ma != M, Nb != N
    if (K != L or M != Mo or N != No or Ka != n or Kb != n or (ta and Ma != -(-M // BLOCK)) or (tb and Nb != -(-N // BLOCK))
            or a_scales.dtype is not SCALE or b_scales.dtype is not SCALE
            or not 0 <= dev == b.get_device() == out.get_device() == a_scales.get_device() == b_scales.get_device() == _args.current_device()):
        return False
    wa, wb, wo, was, wbs = _args.width(a, K), _args.width(b, K), _args.width(out, N), _args.width(a_scales, n), _args.width(b_scales, n)
    if wa < 0 or wb < 0 or wo < 0 or was < 0 or wbs < 0 or wp < 0:
        return False
    _args.done(_args.entry("kda_fp8_matmul")(
        a.data_ptr(), wa, ca, a_scales.data_ptr(), was, ta, b.data_ptr(), wb, cb, b_scales.data_ptr(), wbs, tb, out.data_ptr(), wo, pp, wp,
        dt, M, N, K, _args.stream_handle(None, dev)))
    return True


def quantize(x, q=None, scales=None, qt=None, scales_t=None, tile=False, stream=None) -> None:
    """Writes ``x`` [..., cols] (bf16, fp16 or fp32, rows evenly spaced) in 8 bits to ``q``, shaped
    like x, and ``scales``, and its transpose to ``qt`` [cols, rows] and ``scales_t``, whose blocks
    lie along x's columns; one pass over x does both.  Asynchronous on ``stream`` (default: the
    current torch stream)."""
    if stream is None and _plain_quantize(x, q, scales, qt, scales_t, tile):
        return
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
    if stream is None and _plain_dequantize(q, scales, out):
        return
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
    if stream is None and _plain_matmul(a, a_scales, b, b_scales, out, add):
        return
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

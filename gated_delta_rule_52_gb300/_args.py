"""Argument checks and marshalling shared by the operators around the delta rule (glr,
layer_norm, short_conv): element types, token tensors with strided rows, streams."""
from __future__ import annotations

import contextlib

import torch

from . import kda

DTYPES = {torch.bfloat16: 1, torch.float32: 2, torch.float16: 3}   # kda_dtype


def dtype_code(name, t) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    return code


def ptr(t):
    return None if t is None else t.data_ptr()


def check(name, t, dtype, shape) -> None:
    """A contiguous CUDA tensor of this type and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        kda._check_tensor(name, t, dtype, shape)


def rows(name, t, dtype, shape, lead: int) -> int:
    """Row stride (elements) of a CUDA tensor whose first ``lead`` dimensions index packed
    rows and whose others are one row's contiguous elements.  A slice of a wider tensor
    qualifies; rows that are not evenly spaced do not."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    width = 1
    if t.is_contiguous() or t.numel() == 0:
        for n in shape[lead:]:
            width *= n
        return width
    size, step = t.shape, t.stride()
    for d in range(len(size) - 1, lead - 1, -1):
        if size[d] != 1 and step[d] != width:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        width *= size[d]
    stride, span = None, 0
    for d in range(lead - 1, -1, -1):
        if size[d] == 1:
            continue
        if stride is None:
            stride = step[d]
            span = stride * size[d]
        elif step[d] == span:
            span *= size[d]
        else:
            raise ValueError(f"{name}: rows must be evenly spaced")
    return width if stride is None else stride


def sequences(cu_seqlens) -> int:
    """Number of sequences of cu_seqlens (0 for None)."""
    if cu_seqlens is None:
        return 0
    kda._check_tensor("cu_seqlens", cu_seqlens, torch.int64)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with at least 2 entries")
    return cu_seqlens.numel() - 1


def stream_handle(stream) -> int:
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def on(stream):
    """Allocates what a call returns on the stream that writes it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def done(status: int) -> None:
    if status != kda.KDA_OK:
        raise kda.KDAError(status, kda.status_string(status))

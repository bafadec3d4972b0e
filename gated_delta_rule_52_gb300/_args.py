"""Argument checks and marshalling shared by the operators around the delta rule (glr,
layer_norm, short_conv): element types, token tensors with strided rows, devices, streams.

The library launches on the current device, so a call's tensors and its stream have to be
there: a tensor of another GPU is refused here, before its pointer is used.

A decode step's call costs more on the host than on the GPU, so the checks look at a
contiguous tensor once and take the current stream's handle without building a Stream."""
from __future__ import annotations

import torch

from . import kda

DTYPES = {torch.bfloat16: 1, torch.float32: 2, torch.float16: 3}   # kda_dtype
STATES = {torch.bfloat16: kda.KDA_STATE_BF16, torch.float32: kda.KDA_STATE_FP32}

_entry = {}
current_device = getattr(torch._C, "_cuda_getDevice", None)   # the index, without a Python frame


def entry(name):
    """The library's C entry point."""
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(kda.lib(), name)
    return f


def dtype_code(name, t) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    return code


def device(name, t) -> int:
    """The GPU that a call on this tensor runs on: the current one, where it has to be."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if index != current_device():
        raise ValueError(f"{name} is on cuda:{index}, the current device is cuda:{current_device()}")
    return index


def _elsewhere(name, index, dev):
    raise ValueError(f"{name} must be a CUDA tensor" if index < 0 else f"{name} is on cuda:{index}, the call's device is cuda:{dev}")


def tensor(name, t, dtype, shape, dev: int):
    """Data pointer of a contiguous tensor of this type and shape on this GPU."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        kda._check_tensor(name, t, dtype, shape)
        _elsewhere(name, t.get_device(), dev)
    return t.data_ptr()


def optional(name, t, dtype, shape, dev: int):
    return None if t is None else tensor(name, t, dtype, shape, dev)


def rows(name, t, dtype, shape, lead: int, width: int, dev: int | None = None) -> int:
    """Row stride (elements) of a CUDA tensor (on this GPU, where one is given) whose first
    ``lead`` dimensions index packed rows and whose others are one row's ``width`` contiguous
    elements.  A slice of a wider tensor qualifies; rows that are not evenly spaced do not."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    size = t.shape
    if size != shape:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
    elif t.get_device() != dev:
        _elsewhere(name, t.get_device(), dev)
    if t.is_contiguous() or t.numel() == 0:
        return width
    step, inner = t.stride(), 1
    for d in range(len(size) - 1, lead - 1, -1):
        if size[d] != 1 and step[d] != inner:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        inner *= size[d]
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


def states(initial_state, final_state, shape, dev: int):
    """State dtype code and the data pointers of the states (None where absent)."""
    first = initial_state if initial_state is not None else final_state
    if first is None:
        return kda.KDA_STATE_NONE, None, None
    code = kda.state_dtype_code(initial_state, final_state) if final_state is not initial_state else STATES.get(first.dtype)
    if code is None:
        raise ValueError(f"state dtype must be bf16 or fp32, got {first.dtype}")
    return code, optional("initial_state", initial_state, first.dtype, shape, dev), \
        optional("final_state", final_state, first.dtype, shape, dev)


def sequences(cu_seqlens, dev: int):
    """Number of sequences of cu_seqlens and its data pointer (0 and None for None)."""
    if cu_seqlens is None:
        return 0, None
    kda._check_tensor("cu_seqlens", cu_seqlens, torch.int64)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be 1-D with at least 2 entries")
    if cu_seqlens.get_device() != dev:
        _elsewhere("cu_seqlens", cu_seqlens.get_device(), dev)
    return cu_seqlens.numel() - 1, cu_seqlens.data_ptr()


def stream_handle(stream, dev: int) -> int:
    """Handle of ``stream``, or of the GPU's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the call's device is cuda:{dev}")
    return stream.cuda_stream


def new(stream, t, *shapes):
    """New contiguous tensors of ``t``'s type and device, allocated on the stream that writes
    them (None for a shape of None)."""
    if stream is None:
        return [None if s is None else t.new_empty(s) for s in shapes]
    with torch.cuda.stream(stream):
        return new(None, t, *shapes)


def done(status: int) -> None:
    if status:
        raise kda.KDAError(status, kda.status_string(status))

"""Argument marshalling shared by the bindings of the attention layer's operators (attn.py,
block.py): pointers of checked tensors, the device and stream of a call, workspaces.  The checks
are written for calls of a few microseconds: one look at each property of a tensor."""
from __future__ import annotations

import contextlib

import torch

_F32 = torch.float32
_NO_CONTEXT = contextlib.nullcontext()


def device_index(t, name):
    """The CUDA device of a call's first tensor."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return i


def on(index, stream):
    """The context a call runs in: its device current and, when given, `stream` its current stream, so that
    what the call allocates belongs to the stream it runs on."""
    if stream is None:
        return _NO_CONTEXT if torch.cuda.current_device() == index else torch.cuda.device(index)
    device = torch.device("cuda", index)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def stream_of(index):
    return torch._C._cuda_getCurrentRawStream(index)     # looked up here: a torch without CUDA has none


def _refuse(t, dtype, index, shape, name):
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def ptr(t, dtype, index, shape, name):
    """Pointer of a contiguous tensor (None for None and for an empty one); shape None: any."""
    if t is None:
        return None
    if (shape is not None and t.shape != shape) or t.get_device() != index or t.dtype != dtype or not t.is_contiguous():
        _refuse(t, dtype, index, shape, name)
    return t.data_ptr() or None


def f32(t, index, shape, name):
    return ptr(t, _F32, index, shape, name)


def rows(t, index, n, width, name):
    """Pointer and row stride of an [n, width] fp32 tensor whose rows are contiguous (a column slice of a wider
    array is fine)."""
    if t is None:
        return None, width
    shape = t.shape
    if len(shape) != 2 or shape[0] != n or shape[1] != width or t.get_device() != index or t.dtype != _F32:
        _refuse(t, _F32, index, (n, width), name)
    ld, step = t.stride()
    if n <= 1:
        ld = width
    if (width > 1 and step != 1) or ld < width:
        raise ValueError(f"{name} must have contiguous rows at least {width} floats apart")
    return t.data_ptr() or None, ld


def apart(outputs, inputs, names):
    """Refuses an output that starts where an input or another output does (one tensor given twice); None: not there."""
    given = [p for p in outputs if p]
    if len(set(given)) != len(given) or not set(given).isdisjoint(inputs):
        raise ValueError(f"{names} must not share memory with an input or with one another")


def workspace(ws, need, index):
    """(tensor that keeps it, pointer, bytes)"""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", index))
        return ws, ws.data_ptr(), need
    size = ws.numel() * ws.element_size()
    if ws.get_device() != index:
        raise ValueError(f"workspace must be on cuda:{index}, got {ws.device}")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if size < need:
        raise ValueError(f"workspace needs {need} bytes, got {size}")
    return ws, ws.data_ptr() or None, size

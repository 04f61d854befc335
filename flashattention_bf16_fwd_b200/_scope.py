"""Devices, streams and argument checks that the bindings of the window and cache calls share.

A call of this library takes some microseconds on the GPU for a single short
sequence.  So the usual call (current stream, current device, no workspace given)
goes through the compiled module _fast, which returns None for any other; those,
and calls that are wrong, take the way through ctypes and the checks below.
"""
from __future__ import annotations

import torch

try:
    from . import _fast  # noqa: F401
except ImportError as e:
    raise ImportError("the module _fast is missing or does not fit this torch: build it with "
                      "`python -m flashattention_bf16_fwd_b200.build --force`") from e

_raw_stream = torch._C._cuda_getCurrentRawStream


def call(fn, t, stream, *args):
    """fn(*args, stream) with t's device current and ``stream`` (a torch stream or
    a cudaStream_t; None: the device's current stream) the current stream, so
    that what fn allocates belongs to the stream that uses it."""
    at = t.get_device()
    if at < 0:
        raise ValueError("tensors must live on a CUDA device (the library has no CPU path)")
    if stream is None:
        if at == torch.cuda.current_device():
            return fn(*args, _raw_stream(at))
        with torch.cuda.device(at):
            return fn(*args, _raw_stream(at))
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream)
                  else torch.cuda.default_stream(t.device))
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.stream(stream):
        return fn(*args, stream.cuda_stream)


def same_device(t, *others):
    at = t.get_device()
    for x in others:
        if x is not None and x.get_device() != at:
            raise ValueError("tensors must share one device")


def int32(name, t, *shape):
    """t: a contiguous int32 tensor of this shape (None: any length)."""
    have = t.shape
    if t.dtype is torch.int32 and len(have) == len(shape) and t.is_contiguous():
        for n, want in zip(have, shape):
            if n != want and want is not None:
                break
        else:
            return
    raise ValueError(f"{name} must be a contiguous int32 tensor of shape "
                     f"[{', '.join('*' if n is None else str(n) for n in shape)}], got {t.dtype} {tuple(have)}")


INT_MAX = 2**31 - 1


def count(n) -> int:
    """n, a whole number of any type, as a C int: more than an int holds is as much as the largest one, less than
    nothing is -1."""
    i = int(n)
    if i != n:
        raise ValueError(f"{n} is not a whole number")
    return i if 0 <= i <= INT_MAX else INT_MAX if i > 0 else -1

"""Binding of sliding-window attention with sinks (include/fa_b200_window.h).

Query i sees key j where j <= i and (i - j < window or j < sinks).  The calls
are those of ``fa.attention_fwd`` and ``fa.attention_bwd`` (causal) with that
mask: [B, H, N, d] tensors, bf16 or fp16, d 64 or 128, k and v with H heads or
fewer, every fix_mode.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _scope
from ._scope import _fast
from ._scope import count as _count
from .fa import _check, _elem, _validate, lib

__all__ = ["EXPORTED", "fa_window_bwd_workspace_size", "attention_window_fwd", "attention_window_bwd"]

EXPORTED = ("fa_window_fwd", "fa_window_bwd_workspace_size", "fa_window_bwd")

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
lib.fa_window_fwd.argtypes = [_vp] * 5 + [_i] * 7 + [_f, _i, _i, _vp]
lib.fa_window_bwd_workspace_size.argtypes = [_i] * 7
lib.fa_window_bwd_workspace_size.restype = _sz
lib.fa_window_bwd.argtypes = [_vp] * 10 + [_sz] + [_i] * 7 + [_f, _i, _vp]


@functools.lru_cache(maxsize=256)
def fa_window_bwd_workspace_size(B: int, H: int, Hkv: int, N: int, d: int, window: int, sinks: int) -> int:
    return int(lib.fa_window_bwd_workspace_size(B, H, Hkv, N, d, _count(window), _count(sinks)))


def _valid(q, k, v) -> bool:
    """What _validate asks of q, k and v, in one expression."""
    if not q.dim() == 4 == k.dim():
        return False
    B, H, N, d = q.shape
    shape, dtype, at = k.shape, q.dtype, q.get_device()
    B_, Hkv, N_, d_ = shape
    return (B_ == B and N_ == N and d_ == d and Hkv > 0 and H % Hkv == 0 and shape == v.shape and k.dtype is dtype
            and v.dtype is dtype and k.get_device() == at and v.get_device() == at and q.is_contiguous()
            and k.is_contiguous() and v.is_contiguous())


def attention_window_fwd(q, k, v, window: int, sinks: int = 0, scale: float | None = None, fix_mode: int = 1,
                         stream=None):
    """Allocate O and LSE and run the forward; returns (o, lse)."""
    if stream is None:
        done = _fast.window_fwd(q, k, v, window, sinks, scale, fix_mode)
        if done is not None:
            return done
    if not _valid(q, k, v):
        _validate(q, k, v)
    return _scope.call(_fwd, q, stream, q, k, v, window, sinks, scale, fix_mode, _elem(q))


def _fwd(q, k, v, window, sinks, scale, fix_mode, elem, stream):
    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = q.new_empty((B, H, N), dtype=torch.float32)
    status = lib.fa_window_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, k.shape[1], N,
                               d, _count(window), _count(sinks), d ** -0.5 if scale is None else scale,
                               _count(fix_mode), elem, stream)
    if status:
        _check("fa_window_fwd", status)
    return o, lse


def attention_window_bwd(q, k, v, o, lse, do, window: int, sinks: int = 0, scale: float | None = None, stream=None,
                         workspace=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run the
    backward of attention_window_fwd with the same window and sinks."""
    if stream is None and workspace is None:
        done = _fast.window_bwd(q, k, v, o, lse, do, window, sinks, scale)
        if done is not None:
            return done
    shape, dtype, at = q.shape, q.dtype, q.get_device()
    if not (_valid(q, k, v) and o.shape == shape and do.shape == shape and o.dtype is dtype and do.dtype is dtype
            and o.get_device() == at and do.get_device() == at and o.is_contiguous() and do.is_contiguous()):
        _validate(q, k, v, (o, do))
    if lse.shape != shape[:3] or lse.dtype is not torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    _scope.same_device(q, lse, workspace)
    return _scope.call(_bwd, q, stream, q, k, v, o, lse, do, window, sinks, scale, workspace, _elem(q))


def _bwd(q, k, v, o, lse, do, window, sinks, scale, workspace, elem, stream):
    B, H, N, d = q.shape
    Hkv, window, sinks = k.shape[1], _count(window), _count(sinks)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = q.new_empty(fa_window_bwd_workspace_size(B, H, Hkv, N, d, window, sinks), dtype=torch.uint8)
    status = lib.fa_window_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                               dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.nbytes, B, H,
                               Hkv, N, d, window, sinks, d ** -0.5 if scale is None else scale, elem, stream)
    if status:
        _check("fa_window_bwd", status)
    return dq, dk, dv

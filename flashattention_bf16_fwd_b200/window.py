"""Binding of sliding-window attention with sinks (include/fa_b200_window.h).

Query i sees key j where j <= i and (i - j < window or j < sinks).  The calls
are those of ``fa.attention_fwd`` and ``fa.attention_bwd`` (causal) with that
mask: [B, H, N, d] tensors, bf16 or fp16, d 64 or 128, k and v with H heads or
fewer, every fix_mode.
"""
from __future__ import annotations

import ctypes

import torch

from . import _scope
from .fa import _check, _elem, _shape, _validate, lib

__all__ = ["EXPORTED", "fa_window_bwd_workspace_size", "attention_window_fwd", "attention_window_bwd"]

EXPORTED = ("fa_window_fwd", "fa_window_bwd_workspace_size", "fa_window_bwd")

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
lib.fa_window_fwd.argtypes = [_vp] * 5 + [_i] * 7 + [_f, _i, _i, _vp]
lib.fa_window_bwd_workspace_size.argtypes = [_i] * 7
lib.fa_window_bwd_workspace_size.restype = _sz
lib.fa_window_bwd.argtypes = [_vp] * 10 + [_sz] + [_i] * 7 + [_f, _i, _vp]


def fa_window_bwd_workspace_size(B: int, H: int, Hkv: int, N: int, d: int, window: int, sinks: int) -> int:
    return int(lib.fa_window_bwd_workspace_size(B, H, Hkv, N, d, _scope.count(window), _scope.count(sinks)))


def attention_window_fwd(q, k, v, window: int, sinks: int = 0, scale: float | None = None, fix_mode: int = 1,
                         stream=None):
    """Allocate O and LSE and run the forward; returns (o, lse)."""
    _validate(q, k, v)
    B, H, N, d = _shape(q)
    with _scope.scope(q, stream):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
        _check("fa_window_fwd", lib.fa_window_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, int(k.shape[1]), N, d,
            _scope.count(window), _scope.count(sinks), d ** -0.5 if scale is None else float(scale), int(fix_mode),
            _elem(q), _scope.current()))
    return o, lse


def attention_window_bwd(q, k, v, o, lse, do, window: int, sinks: int = 0, scale: float | None = None, stream=None,
                         workspace=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run the
    backward of attention_window_fwd with the same window and sinks."""
    _validate(q, k, v, (o, do))
    B, H, N, d = _shape(q)
    if lse.shape != (B, H, N) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    _scope.same_device(q, lse, workspace)
    Hkv = int(k.shape[1])
    with _scope.scope(q, stream):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        if workspace is None:
            workspace = torch.empty(fa_window_bwd_workspace_size(B, H, Hkv, N, d, window, sinks), dtype=torch.uint8,
                                    device=q.device)
        _check("fa_window_bwd", lib.fa_window_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), B, H, Hkv,
            N, d, _scope.count(window), _scope.count(sinks), d ** -0.5 if scale is None else float(scale), _elem(q),
            _scope.current()))
    return dq, dk, dv

"""Binding of the paged key/value cache (include/fa_b200_cache.h): attention of
one new token per sequence, writing tokens, and the page operators.

A cache is four kinds of tensors that the caller owns, all on the GPU:

* ``k_pages``, ``v_pages``: [P, Hkv, page, d] bf16 or fp16, one layer; the page
  operators also take all layers at once, [L, P, Hkv, page, d],
* ``table``: int32 [S, M], entry i of row s the page of tokens i*page and on,
* ``lens``: int32 [S], 0 for an empty slot,
* ``refs``: int32 [P], how many table entries name a page, 0 for a free one.

A decoding step::

    cache_reserve(refs, table, lens, ones, page)          # lens += 1, pages where one begins
    for layer in range(L):
        cache_append(k[layer], v[layer], k_pages[layer], v_pages[layer], table, lens)
        o, lse = attention_decode(q[layer], k_pages[layer], v_pages[layer], table, lens)

Nothing synchronises: lengths, pages and outcomes stay on the device (a call
that found one out of range is reported by ``fa.fa_check_device_error``), and a
step can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

from . import _scope
from .fa import _check, _elem, lib

__all__ = ["EXPORTED", "fa_decode_workspace_size", "fa_cache_workspace_size", "attention_decode", "cache_append",
           "cache_reserve", "cache_fork", "cache_free", "cache_compact"]

EXPORTED = ("fa_decode_workspace_size", "fa_decode", "fa_cache_append", "fa_cache_reserve", "fa_cache_workspace_size",
            "fa_cache_fork", "fa_cache_free", "fa_cache_compact")

_vp, _i, _f, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
lib.fa_decode_workspace_size.argtypes = [_i] * 4
lib.fa_decode_workspace_size.restype = _sz
lib.fa_decode.argtypes = [_vp] * 8 + [_sz] + [_i] * 7 + [_ll, _i, _i, _f, _i, _vp]
lib.fa_cache_append.argtypes = [_vp] * 7 + [_i] * 7 + [_ll, _ll, _vp]
lib.fa_cache_reserve.argtypes = [_vp] * 5 + [_i] * 4 + [_vp]
lib.fa_cache_workspace_size.argtypes = [_i, _i]
lib.fa_cache_workspace_size.restype = _sz
lib.fa_cache_fork.argtypes = [_vp] * 9 + [_sz] + [_i] * 8 + [_vp]
lib.fa_cache_free.argtypes = [_vp] * 4 + [_i] * 5 + [_vp]
lib.fa_cache_compact.argtypes = [_vp] * 7 + [_sz] + [_i] * 7 + [_vp]


def fa_decode_workspace_size(S: int, H: int, Hkv: int, d: int) -> int:
    return int(lib.fa_decode_workspace_size(S, H, Hkv, d))


def fa_cache_workspace_size(S: int, P: int) -> int:
    return int(lib.fa_cache_workspace_size(S, P))


def _pages(k_pages, v_pages, layers: bool):
    """(L, P, Hkv, page, d) of a cache; L is 1 where there is one layer."""
    dims = (4, 5) if layers else (4,)
    if k_pages.dim() not in dims or v_pages.shape != k_pages.shape:
        raise ValueError(f"k_pages and v_pages must be {'[P, Hkv, page, d] or [L, P, Hkv, page, d]' if layers else '[P, Hkv, page, d]'}, "
                         f"got {tuple(k_pages.shape)}, {tuple(v_pages.shape)}")
    _elem(k_pages)
    if v_pages.dtype != k_pages.dtype or not k_pages.is_contiguous() or not v_pages.is_contiguous():
        raise ValueError("k_pages and v_pages must share one dtype and be contiguous")
    shape = tuple(k_pages.shape)
    return shape if len(shape) == 5 else (1,) + shape


def _rows(name, t, heads, d, dtype):
    """Elements between the tokens of t [*, heads, d]; a token's heads are contiguous."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d or t.dtype != dtype:
        raise ValueError(f"{name} must be [*, {heads}, {d}] of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    if t.shape[0] == 0:
        return heads * d
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"the heads of a token in {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else heads * d


def attention_decode(q, k_pages, v_pages, table, lens, window: int | None = None, sinks: int = 0,
                     scale: float | None = None, stream=None, workspace=None):
    """Attention of the newest token of each sequence, q [S, H, d] (the rows of
    a fused projection are taken as they are), over the cache; returns
    (o [S, H, d], lse [S, H]).  ``window`` None or 0 shows every key; otherwise
    the last ``window`` keys and the first ``sinks``."""
    if q.dim() != 3:
        raise ValueError("q must be [S, H, d]")
    _, P, Hkv, page, d = _pages(k_pages, v_pages, False)
    S, H = int(q.shape[0]), int(q.shape[1])
    if H % Hkv != 0 or H == 0:
        raise ValueError(f"the {Hkv} key/value heads must divide the {H} query heads")
    stride = _rows("q", q, H, d, k_pages.dtype)
    _scope.int32("table", table, (S, None))
    _scope.int32("lens", lens, (S,))
    _scope.same_device(q, k_pages, v_pages, table, lens, workspace)
    with _scope.scope(q, stream):
        o = torch.empty((S, H, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((S, H), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.empty(fa_decode_workspace_size(S, H, Hkv, d), dtype=torch.uint8, device=q.device)
        _check("fa_decode", lib.fa_decode(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), o.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), S, H, Hkv, d, P, page,
            int(table.shape[1]), stride, _scope.count(window or 0), _scope.count(sinks),
            d ** -0.5 if scale is None else float(scale),
            _elem(q), _scope.current()))
    return o, lse


def cache_append(k, v, k_pages, v_pages, table, lens, cu=None, stream=None):
    """Write the newest tokens, k and v [T, Hkv, d], of each sequence into one
    layer's pages: tokens cu[s] .. cu[s+1]-1 are the last ones of sequence s
    (``cu`` None: one token per sequence).  ``lens`` counts them already."""
    _, P, Hkv, page, d = _pages(k_pages, v_pages, False)
    ks, vs = _rows("k", k, Hkv, d, k_pages.dtype), _rows("v", v, Hkv, d, k_pages.dtype)
    T, S = int(k.shape[0]), int(table.shape[0])
    if v.shape[0] != T or (cu is None and T != S):
        raise ValueError(f"k and v must have one row per token ({S} sequences), got {T} and {v.shape[0]}")
    _scope.int32("table", table, (S, None))
    _scope.int32("lens", lens, (S,))
    if cu is not None:
        _scope.int32("cu", cu, (S + 1,))
    _scope.same_device(k_pages, v_pages, k, v, table, lens, cu)
    with _scope.scope(k_pages, stream):
        if T == 0:
            return
        _check("fa_cache_append", lib.fa_cache_append(
            k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(),
            None if cu is None else cu.data_ptr(), T, S, Hkv, d, P, page, int(table.shape[1]), ks, vs,
            _scope.current()))


def _tables(refs, table, lens, P=None):
    _scope.int32("refs", refs, (P,))
    _scope.int32("table", table, (None, None))
    _scope.int32("lens", lens, (int(table.shape[0]),))
    _scope.same_device(refs, table, lens)
    return int(refs.shape[0]), int(table.shape[0]), int(table.shape[1])


def cache_reserve(refs, table, lens, add, page: int, stream=None):
    """lens += add, with pages for the new tokens.  Returns ``missing``, int32
    [1] on the device: 0 when done, the number of pages lacking (nothing is
    changed then), or -1 (a length or an entry of add is out of range)."""
    P, S, M = _tables(refs, table, lens)
    _scope.int32("add", add, (S,))
    _scope.same_device(refs, add)
    with _scope.scope(refs, stream):
        missing = torch.empty(1, dtype=torch.int32, device=refs.device)
        _check("fa_cache_reserve", lib.fa_cache_reserve(
            refs.data_ptr(), table.data_ptr(), lens.data_ptr(), add.data_ptr(), missing.data_ptr(), S, P, int(page), M,
            _scope.current()))
    return missing


def cache_fork(k_pages, v_pages, refs, table, lens, src, dst, stream=None, workspace=None):
    """Sequence dst[f] (an empty slot) becomes a copy of sequence src[f]: full
    pages are shared, a last page that is not full is copied.  Returns
    ``missing`` as in cache_reserve."""
    L, P, Hkv, page, d = _pages(k_pages, v_pages, True)
    _, S, M = _tables(refs, table, lens, P)
    _scope.int32("src", src, (None,))
    F = int(src.shape[0])
    _scope.int32("dst", dst, (F,))
    _scope.same_device(refs, k_pages, v_pages, src, dst, workspace)
    with _scope.scope(refs, stream):
        missing = torch.empty(1, dtype=torch.int32, device=refs.device)
        if workspace is None:
            workspace = torch.empty(fa_cache_workspace_size(S, P), dtype=torch.uint8, device=refs.device)
        _check("fa_cache_fork", lib.fa_cache_fork(
            k_pages.data_ptr(), v_pages.data_ptr(), refs.data_ptr(), table.data_ptr(), lens.data_ptr(), src.data_ptr(),
            dst.data_ptr(), missing.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), F,
            L, S, Hkv, d, P, page, M, _scope.current()))
    return missing


def cache_free(refs, table, lens, seqs, page: int, stream=None):
    """End the sequences ``seqs`` (int32 [F]): their pages' counts fall by 1,
    their table entries become -1 and their lengths 0."""
    P, S, M = _tables(refs, table, lens)
    _scope.int32("seqs", seqs, (None,))
    _scope.same_device(refs, seqs)
    with _scope.scope(refs, stream):
        _check("fa_cache_free", lib.fa_cache_free(
            refs.data_ptr(), table.data_ptr(), lens.data_ptr(), seqs.data_ptr(), int(seqs.shape[0]), S, P, int(page), M,
            _scope.current()))


def cache_compact(k_pages, v_pages, refs, table, lens, stream=None, workspace=None):
    """Move the pages in use to the numbers 0 .. live-1 (in all layers, with
    tables and counts).  Returns ``live``, int32 [1] on the device."""
    L, P, Hkv, page, d = _pages(k_pages, v_pages, True)
    _, S, M = _tables(refs, table, lens, P)
    _scope.same_device(refs, k_pages, v_pages, workspace)
    with _scope.scope(refs, stream):
        live = torch.empty(1, dtype=torch.int32, device=refs.device)
        if workspace is None:
            workspace = torch.empty(fa_cache_workspace_size(S, P), dtype=torch.uint8, device=refs.device)
        _check("fa_cache_compact", lib.fa_cache_compact(
            k_pages.data_ptr(), v_pages.data_ptr(), refs.data_ptr(), table.data_ptr(), lens.data_ptr(), live.data_ptr(),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), L, S, Hkv, d, P, page, M,
            _scope.current()))
    return live

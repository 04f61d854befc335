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
step can be captured into a CUDA graph.  Calls on one cache are put in order by
the caller: by one stream, and among Python threads by a lock (a call lets other
threads run while it launches).
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _scope
from ._scope import _fast
from ._scope import count as _count
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


@functools.lru_cache(maxsize=256)
def fa_decode_workspace_size(S: int, H: int, Hkv: int, d: int) -> int:
    return int(lib.fa_decode_workspace_size(S, H, Hkv, d))


@functools.lru_cache(maxsize=256)
def fa_cache_workspace_size(S: int, P: int) -> int:
    return int(lib.fa_cache_workspace_size(S, P))


def _pages(k_pages, v_pages, layers: bool):
    """The shape of a cache, (P, Hkv, page, d) or, with layers, (L, P, Hkv, page, d)."""
    shape = k_pages.shape
    if (len(shape) == 4 or (layers and len(shape) == 5)) and shape == v_pages.shape and (
            k_pages.dtype is v_pages.dtype and k_pages.is_contiguous() and v_pages.is_contiguous()):
        return shape if len(shape) == 5 or not layers else (1, *shape)
    if shape != v_pages.shape or len(shape) not in ((4, 5) if layers else (4,)):
        raise ValueError(f"k_pages and v_pages must be {'[P, Hkv, page, d] or [L, P, Hkv, page, d]' if layers else '[P, Hkv, page, d]'}, "
                         f"got {tuple(shape)}, {tuple(v_pages.shape)}")
    raise ValueError("k_pages and v_pages must share one dtype and be contiguous")


def _rows(name, t, heads, d, dtype):
    """Elements between the tokens of t [*, heads, d]; a token's heads are contiguous."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or t.dtype is not dtype:
        raise ValueError(f"{name} must be [*, {heads}, {d}] of {dtype}, got {tuple(shape)} of {t.dtype}")
    if t.is_contiguous():
        return heads * d
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"the heads of a token in {name} must be contiguous")
    return t.stride(0) if shape[0] > 1 else heads * d


def _table(table, lens, S=None):
    """(S, M) of the table; lens has S entries."""
    shape = table.shape
    if not (len(shape) == 2 and lens.shape == shape[:1] and (S is None or S == shape[0]) and table.dtype is torch.int32
            and lens.dtype is torch.int32 and table.is_contiguous() and lens.is_contiguous()):
        _scope.int32("table", table, S, None)
        _scope.int32("lens", lens, table.shape[0])
    return shape


def attention_decode(q, k_pages, v_pages, table, lens, window: int | None = None, sinks: int = 0,
                     scale: float | None = None, stream=None, workspace=None):
    """Attention of the newest token of each sequence, q [S, H, d] (the rows of
    a fused projection are taken as they are), over the cache; returns
    (o [S, H, d], lse [S, H]).  ``window`` None or 0 shows every key; otherwise
    the last ``window`` keys and the first ``sinks``."""
    if stream is None and workspace is None:
        done = _fast.decode(q, k_pages, v_pages, table, lens, window, sinks, scale)
        if done is not None:
            return done
    if q.dim() != 3:
        raise ValueError("q must be [S, H, d]")
    P, Hkv, page, d = _pages(k_pages, v_pages, False)
    S, H, _ = q.shape
    if Hkv == 0 or H == 0 or H % Hkv:
        raise ValueError(f"the {Hkv} key/value heads must divide the {H} query heads")
    stride = _rows("q", q, H, d, k_pages.dtype)
    M = _table(table, lens, S)[1]
    at = q.get_device()
    if not (at == k_pages.get_device() == v_pages.get_device() == table.get_device() == lens.get_device()
            and (workspace is None or workspace.get_device() == at)):
        raise ValueError("tensors must share one device")
    return _scope.call(_decode, q, stream, q, k_pages, v_pages, table, lens, workspace,
                       (S, H, Hkv, d, P, page, M, stride, _count(window or 0), _count(sinks),
                        d ** -0.5 if scale is None else scale, _elem(q)))


def _decode(q, k_pages, v_pages, table, lens, workspace, sizes, stream):
    S, H, Hkv, d = sizes[:4]
    o = torch.empty_like(q) if q.is_contiguous() else q.new_empty((S, H, d))
    lse = q.new_empty((S, H), dtype=torch.float32)
    if workspace is None:
        workspace = q.new_empty(fa_decode_workspace_size(S, H, Hkv, d), dtype=torch.uint8)
    status = lib.fa_decode(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(),
                           o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, *sizes, stream)
    if status:
        _check("fa_decode", status)
    return o, lse


def cache_append(k, v, k_pages, v_pages, table, lens, cu=None, stream=None):
    """Write the newest tokens, k and v [T, Hkv, d], of each sequence into one
    layer's pages: tokens cu[s] .. cu[s+1]-1 are the last ones of sequence s
    (``cu`` None: one token per sequence).  ``lens`` counts them already."""
    if stream is None and _fast.append(k, v, k_pages, v_pages, table, lens, cu):
        return
    P, Hkv, page, d = _pages(k_pages, v_pages, False)
    dtype = k_pages.dtype
    _elem(k_pages)
    ks, vs = _rows("k", k, Hkv, d, dtype), _rows("v", v, Hkv, d, dtype)
    S, M = _table(table, lens)
    T = k.shape[0]
    if v.shape[0] != T or (cu is None and T != S):
        raise ValueError(f"k and v must have one row per token ({S} sequences), got {T} and {v.shape[0]}")
    at = k_pages.get_device()
    if cu is not None:
        _scope.int32("cu", cu, S + 1)
        _scope.same_device(k_pages, cu)
    if not at == v_pages.get_device() == k.get_device() == v.get_device() == table.get_device() == lens.get_device():
        raise ValueError("tensors must share one device")
    if T == 0:
        return
    status = _scope.call(lib.fa_cache_append, k_pages, stream, k.data_ptr(), v.data_ptr(), k_pages.data_ptr(),
                         v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), None if cu is None else cu.data_ptr(), T, S,
                         Hkv, d, P, page, M, ks, vs)
    if status:
        _check("fa_cache_append", status)


def _page_tables(refs, table, lens, P=None):
    """(P, S, M) of a cache's tables."""
    if refs.dim() != 1 or refs.dtype is not torch.int32 or not refs.is_contiguous() or (P is not None and refs.shape[0] != P):
        _scope.int32("refs", refs, P)
    S, M = _table(table, lens)
    if not refs.get_device() == table.get_device() == lens.get_device():
        raise ValueError("tensors must share one device")
    return refs.shape[0], S, M


def cache_reserve(refs, table, lens, add, page: int, stream=None):
    """lens += add, with pages for the new tokens.  Returns ``missing``, int32
    [1] on the device: 0 when done, the number of pages lacking (nothing is
    changed then), or -1 (a length or an entry of add is out of range)."""
    if stream is None:
        missing = _fast.reserve(refs, table, lens, add, page)
        if missing is not None:
            return missing
    P, S, M = _page_tables(refs, table, lens)
    _scope.int32("add", add, S)
    _scope.same_device(refs, add)
    return _scope.call(_reserve, refs, stream, refs, table, lens, add, (S, P, _count(page), M))


def _reserve(refs, table, lens, add, sizes, stream):
    missing = refs.new_empty(1)
    status = lib.fa_cache_reserve(refs.data_ptr(), table.data_ptr(), lens.data_ptr(), add.data_ptr(), missing.data_ptr(),
                                  *sizes, stream)
    if status:
        _check("fa_cache_reserve", status)
    return missing


def cache_fork(k_pages, v_pages, refs, table, lens, src, dst, stream=None, workspace=None):
    """Sequence dst[f] (an empty slot) becomes a copy of sequence src[f]: full
    pages are shared, a last page that is not full is copied.  Returns
    ``missing`` as in cache_reserve."""
    if stream is None and workspace is None:
        missing = _fast.fork(k_pages, v_pages, refs, table, lens, src, dst)
        if missing is not None:
            return missing
    L, P, Hkv, page, d = _pages(k_pages, v_pages, True)
    _elem(k_pages)
    _, S, M = _page_tables(refs, table, lens, P)
    _scope.int32("src", src, None)
    _scope.int32("dst", dst, src.shape[0])
    _scope.same_device(refs, k_pages, v_pages, src, dst, workspace)
    return _scope.call(_fork, refs, stream, k_pages, v_pages, refs, table, lens, src, dst, workspace,
                       (src.shape[0], L, S, Hkv, d, P, page, M))


def _fork(k_pages, v_pages, refs, table, lens, src, dst, workspace, sizes, stream):
    missing = refs.new_empty(1)
    if workspace is None:
        workspace = refs.new_empty(fa_cache_workspace_size(sizes[2], sizes[5]), dtype=torch.uint8)
    status = lib.fa_cache_fork(k_pages.data_ptr(), v_pages.data_ptr(), refs.data_ptr(), table.data_ptr(), lens.data_ptr(),
                               src.data_ptr(), dst.data_ptr(), missing.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                               *sizes, stream)
    if status:
        _check("fa_cache_fork", status)
    return missing


def cache_free(refs, table, lens, seqs, page: int, stream=None):
    """End the sequences ``seqs`` (int32 [F]): their pages' counts fall by 1,
    their table entries become -1 and their lengths 0."""
    if stream is None and _fast.free(refs, table, lens, seqs, page):
        return
    P, S, M = _page_tables(refs, table, lens)
    _scope.int32("seqs", seqs, None)
    _scope.same_device(refs, seqs)
    status = _scope.call(lib.fa_cache_free, refs, stream, refs.data_ptr(), table.data_ptr(), lens.data_ptr(),
                         seqs.data_ptr(), seqs.shape[0], S, P, _count(page), M)
    if status:
        _check("fa_cache_free", status)


def cache_compact(k_pages, v_pages, refs, table, lens, stream=None, workspace=None):
    """Move the pages in use to the numbers 0 .. live-1 (in all layers, with
    tables and counts).  Returns ``live``, int32 [1] on the device."""
    if stream is None and workspace is None:
        live = _fast.compact(k_pages, v_pages, refs, table, lens)
        if live is not None:
            return live
    L, P, Hkv, page, d = _pages(k_pages, v_pages, True)
    _elem(k_pages)
    _, S, M = _page_tables(refs, table, lens, P)
    _scope.same_device(refs, k_pages, v_pages, workspace)
    return _scope.call(_compact, refs, stream, k_pages, v_pages, refs, table, lens, workspace,
                       (L, S, Hkv, d, P, page, M))


def _compact(k_pages, v_pages, refs, table, lens, workspace, sizes, stream):
    live = refs.new_empty(1)
    if workspace is None:
        workspace = refs.new_empty(fa_cache_workspace_size(sizes[1], sizes[4]), dtype=torch.uint8)
    status = lib.fa_cache_compact(k_pages.data_ptr(), v_pages.data_ptr(), refs.data_ptr(), table.data_ptr(),
                                  lens.data_ptr(), live.data_ptr(), workspace.data_ptr(), workspace.nbytes, *sizes, stream)
    if status:
        _check("fa_cache_compact", status)
    return live

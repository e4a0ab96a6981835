"""Decoding with a paged K/V cache: the Python side of the decode calls in include/stem.h.

    cache = PagedCache.alloc(num_pages, Hkv, D, block, "q4", table, device)
    stem_cache_append(cache, k, v, pos)                  # K, V [nseq, Hkv, T, D] of new tokens
    budget, kcap = stem_decode_budget(cache.max_blocks, method, device)
    out, lse, sel_idx, sel_cnt = stem_decode(cache, q, lens, budget, kcap, method)

A page holds one selection block of one sequence; the caller hands pages out by writing `table`
[nseq, max_blocks]. Calls are asynchronous on `stream` (default: torch's current stream of the
cache's device) and make that device current while they launch. Tensors that a call makes itself
(outputs, workspace) are allocated on torch's current stream: a caller that passes another stream
passes its own outputs and workspace too, or orders the two streams itself.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import stem as _stem
from .stem import (STEM_BF16, STEM_F32, STEM_KV_BF16, STEM_KV_Q4, STEM_KV_Q8, STEM_SHARE_GROUP,
                   STEM_SHARE_HEAD, STEM_VSUM_MAX, STEM_VSUM_MEAN, StemError, make_method,
                   stem_budget_m, stem_cache_t, stem_decode_args_t, stem_method_t)

_lib = _stem.lib()
_FORMATS = {"bf16": STEM_KV_BF16, "q8": STEM_KV_Q8, "q4": STEM_KV_Q4}
_VSUMS = {"mean": STEM_VSUM_MEAN, "max": STEM_VSUM_MAX}
_SHARES = {"head": STEM_SHARE_HEAD, "group": STEM_SHARE_GROUP}
_ATTN = {k: stem_method_t(share=v) for k, v in _SHARES.items()}  # all that the attention reads
_Strides = ctypes.c_int64 * 3

__all__ = ["PagedCache", "stem_cache_page_bytes", "stem_cache_append", "stem_cache_read",
           "stem_decode_budget", "stem_decode_workspace_size", "stem_decode_select",
           "stem_decode_attn", "stem_decode", "make_method", "StemError"]


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device) -> None:
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    raise ValueError(f"{name} must be contiguous")


@functools.lru_cache(maxsize=None)
def stem_cache_page_bytes(D: int, block: int, fmt: str) -> int:
    """Bytes of the record of one (page, kv head); 0 if the library does not support the shape."""
    return int(_lib.stem_cache_page_bytes(D, block, _FORMATS[fmt]))


class PagedCache:
    """A paged cache over tensors that the caller owns:

    pages [num_pages, Hkv, stem_cache_page_bytes(D, block, fmt)] uint8, kbar [num_pages, Hkv, D]
    and vnorm [num_pages, Hkv] float32, table [nseq, max_blocks] int32, all contiguous on one CUDA
    device. fmt: "bf16", "q8" or "q4"; vsum: "mean" or "max" (the block summary of the V norms).
    """

    __slots__ = ("pages", "kbar", "vnorm", "table", "block", "fmt", "vsum", "device", "D", "Hkv",
                 "nseq", "max_blocks", "c", "at")

    def __init__(self, pages, kbar, vnorm, table, block: int, fmt: str, vsum: str = "mean"):
        if kbar.dim() != 3 or table.dim() != 2:
            raise ValueError("kbar must be [num_pages, Hkv, D] and table [nseq, max_blocks]")
        if fmt not in _FORMATS:
            raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt!r}")
        if vsum not in _VSUMS:
            raise ValueError(f"vsum must be one of {sorted(_VSUMS)}, got {vsum!r}")
        n, Hkv, D = kbar.shape
        dev = pages.device
        size = stem_cache_page_bytes(D, block, fmt)
        if size == 0:
            raise ValueError(f"D and block must be 64 or 128, got {D} and {block}")
        if dev.type != "cuda":
            raise ValueError(f"the cache must be on a CUDA device, got {dev}")
        _need(pages, "pages", torch.uint8, (n, Hkv, size), dev)
        _need(kbar, "kbar", torch.float32, (n, Hkv, D), dev)
        _need(vnorm, "vnorm", torch.float32, (n, Hkv), dev)
        _need(table, "table", torch.int32, table.shape, dev)
        nseq, max_blocks = table.shape
        self.pages, self.kbar, self.vnorm, self.table = pages, kbar, vnorm, table
        self.block, self.fmt, self.vsum, self.device = block, fmt, vsum, dev
        self.D, self.Hkv, self.nseq, self.max_blocks = D, Hkv, nseq, max_blocks
        self.c = stem_cache_t(pages.data_ptr(), kbar.data_ptr(), vnorm.data_ptr(),
                              table.data_ptr(), n, Hkv, D, block, _FORMATS[fmt], nseq, max_blocks,
                              _VSUMS[vsum])
        self.at = ctypes.addressof(self.c)

    @classmethod
    def alloc(cls, num_pages: int, Hkv: int, D: int, block: int, fmt: str, table: torch.Tensor,
              vsum: str = "mean") -> "PagedCache":
        """A cache with new buffers (zeroed) on the device of `table`."""
        dev = table.device
        if fmt not in _FORMATS:
            raise ValueError(f"fmt must be one of {sorted(_FORMATS)}, got {fmt!r}")
        size = stem_cache_page_bytes(D, block, fmt)
        return cls(torch.zeros((num_pages, Hkv, size), dtype=torch.uint8, device=dev),
                   torch.zeros((num_pages, Hkv, D), dtype=torch.float32, device=dev),
                   torch.zeros((num_pages, Hkv), dtype=torch.float32, device=dev), table, block,
                   fmt, vsum)


def _launch(fn, cache: PagedCache, stream, *args):
    """fn(*args, stream) with the cache's device current."""
    dev = cache.device
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the cache on {dev}")
    else:
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc:
        raise StemError(rc, fn.__name__)


def _status(status, dev):
    if status is None:
        return None
    _need(status, "status", torch.int32, (1,), dev)
    return status.data_ptr()


# ------------------------------------------------------------------ the cache


def _rows(fn, cache, k, v, pos, count, status, stream):
    dev = cache.device
    if k.dim() != 4 or k.shape[0] != cache.nseq or k.shape[1] != cache.Hkv or \
            k.shape[3] != cache.D:
        raise ValueError(f"k must be [{cache.nseq}, {cache.Hkv}, T, {cache.D}], got "
                         f"{tuple(k.shape)}")
    T = k.shape[2]
    strides = k.stride()
    if v.shape != k.shape or v.dtype is not k.dtype or v.stride() != strides:
        raise ValueError("k and v must have the same shape, dtype and strides")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on the cache's device {dev}")
    if strides[3] != 1:
        raise ValueError("k and v must be contiguous in their last dimension")
    if k.dtype is torch.bfloat16:
        code = STEM_BF16
    elif k.dtype is torch.float32:
        code = STEM_F32
    else:
        raise TypeError(f"k and v must be bfloat16 or float32, got {k.dtype}")
    _need(pos, "pos", torch.int32, (cache.nseq,), dev)
    if count is not None:
        _need(count, "count", torch.int32, (cache.nseq,), dev)
    _launch(fn, cache, stream, cache.at, k.data_ptr(), v.data_ptr(), code, T,
            _Strides(*strides[:3]), pos.data_ptr(), None if count is None else count.data_ptr(),
            _status(status, dev))


def stem_cache_append(cache: PagedCache, k, v, pos, count=None, status=None, stream=None) -> None:
    """Write K and V rows k, v [nseq, Hkv, T, D] (bf16 or f32, any strides with a contiguous last
    dimension and rows on 16-byte boundaries) as tokens pos[s] .. pos[s] + count[s] - 1 of each
    sequence (count None: all T), quantised to the cache's format, and summarise the blocks that
    this completes."""
    _rows(_lib.stem_cache_append, cache, k, v, pos, count, status, stream)


def stem_cache_read(cache: PagedCache, pos, count=None, k=None, v=None, T: Optional[int] = None,
                    dtype=torch.bfloat16, status=None, stream=None):
    """The values that tokens pos[s] .. pos[s] + count[s] - 1 stand for: (k, v) [nseq, Hkv, T, D],
    given, or made with T rows (rows past count then hold zeros). Rows past count of given tensors
    are left as they were."""
    if (k is None) != (v is None):
        raise ValueError("give both of k and v, or neither")
    if k is None:
        if T is None:
            raise ValueError("T is needed when k and v are not given")
        k = torch.zeros((cache.nseq, cache.Hkv, T, cache.D), dtype=dtype, device=cache.device)
        v = torch.zeros_like(k)
    _rows(_lib.stem_cache_read, cache, k, v, pos, count, status, stream)
    return k, v


# ------------------------------------------------------------------ decode


def stem_decode_budget(max_blocks: int, method: stem_method_t, device):
    """(budget [max_blocks] int32 on `device`, kcap): k(i) of the method's schedule for a query in
    block i, and its largest value. Made once per method and context size."""
    k, _ = stem_budget_m(max_blocks, method)
    return k.to(device), max(int(k.max()), 1)


def stem_decode_workspace_size(cache: PagedCache, R: int, Hq: int, kcap: int) -> int:
    """Workspace bytes of a decode call of R rows; one workspace per call that may overlap another."""
    return _workspace_size(cache.device.index, cache.fmt, cache.D, cache.block, cache.Hkv,
                           cache.max_blocks, R, Hq, kcap)


@functools.lru_cache(maxsize=4096)
def _workspace_size(device, fmt, D, block, Hkv, max_blocks, R, Hq, kcap):
    c = stem_cache_t(None, None, None, None, 1, Hkv, D, block, _FORMATS[fmt], 1, max_blocks, 0)
    with torch.cuda.device(device):
        return int(_lib.stem_decode_workspace_size(ctypes.addressof(c), R, Hq, kcap))


def _decode(fn, cache, q, lens, rows, budget, kcap, method, sel_idx, sel_cnt, out, lse, workspace,
            status, stream):
    dev = cache.device
    if q.dim() != 3 or q.shape[2] != cache.D:
        raise ValueError(f"q must be [R, Hq, {cache.D}], got {tuple(q.shape)}")
    R, Hq, D = shape = q.shape
    _need(q, "q", torch.bfloat16, shape, dev)
    _need(lens, "lens", torch.int32, (R,), dev)
    if rows is not None:
        _need(rows, "rows", torch.int32, (R,), dev)
        rows = rows.data_ptr()
    if budget is not None:
        _need(budget, "budget", torch.int32, (cache.max_blocks,), dev)
        budget = budget.data_ptr()
    _need(sel_idx, "sel_idx", torch.int32, (R, Hq, kcap), dev)
    _need(sel_cnt, "sel_cnt", torch.int32, (R, Hq), dev)
    if out is None:  # a selection alone needs no workspace
        at, size, out = None, 0, None
    else:
        _need(out, "out", torch.bfloat16, shape, dev)
        out = out.data_ptr()
        if workspace is None:
            workspace = torch.empty(stem_decode_workspace_size(cache, R, Hq, kcap),
                                    dtype=torch.uint8, device=dev)
        elif workspace.device != dev or workspace.dtype is not torch.uint8 or \
                not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor on the cache's device")
        at, size = workspace.data_ptr(), workspace.numel()
    if lse is not None:
        _need(lse, "lse", torch.float32, (R, Hq), dev)
        lse = lse.data_ptr()
    a = stem_decode_args_t(cache.at, q.data_ptr(), rows, lens.data_ptr(), budget, R, Hq, kcap,
                           STEM_BF16, ctypes.addressof(method), sel_idx.data_ptr(),
                           sel_cnt.data_ptr(), out, lse, at, size, _status(status, dev))
    _launch(fn, cache, stream, ctypes.addressof(a))


def _lists(q, kcap, sel_idx, sel_cnt):
    if (sel_idx is None) != (sel_cnt is None):
        raise ValueError("give both of sel_idx and sel_cnt, or neither")
    if sel_idx is None:
        R, Hq = q.shape[:2]
        sel_idx = torch.empty((R, Hq, kcap), dtype=torch.int32, device=q.device)
        sel_cnt = torch.empty((R, Hq), dtype=torch.int32, device=q.device)
    return sel_idx, sel_cnt


def stem_decode_select(cache: PagedCache, q, lens, budget, kcap: int, method: stem_method_t,
                       rows=None, sel_idx=None, sel_cnt=None, status=None, stream=None):
    """Kept blocks of query tokens q [R, Hq, D] (bf16) that see lens[r] tokens of sequence rows[r]
    (None: sequence r). Returns (sel_idx [R, Hq, kcap], ascending, -1 past the count, and sel_cnt
    [R, Hq])."""
    sel_idx, sel_cnt = _lists(q, kcap, sel_idx, sel_cnt)
    _decode(_lib.stem_decode_select, cache, q, lens, rows, budget, kcap, method, sel_idx, sel_cnt,
            None, None, None, status, stream)
    return sel_idx, sel_cnt


def stem_decode_attn(cache: PagedCache, q, lens, sel_idx, sel_cnt, share: str = "head", rows=None,
                     out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of query tokens q [R, Hq, D] over the kept blocks sel_idx [R, Hq, kcap], sel_cnt
    [R, Hq]. share "group": the query heads of a kv head have one list, that of the first. Returns
    (out [R, Hq, D] bf16, lse [R, Hq] float32)."""
    if share not in _SHARES:
        raise ValueError(f"share must be one of {sorted(_SHARES)}, got {share!r}")
    if sel_idx.dim() != 3:
        raise ValueError(f"sel_idx must be [R, Hq, kcap], got {tuple(sel_idx.shape)}")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    _decode(_lib.stem_decode_attn, cache, q, lens, rows, None, sel_idx.shape[2], _ATTN[share],
            sel_idx, sel_cnt, out, lse, workspace, status, stream)
    return out, lse


def stem_decode(cache: PagedCache, q, lens, budget, kcap: int, method: stem_method_t, rows=None,
                out=None, lse=None, sel_idx=None, sel_cnt=None, workspace=None, status=None,
                stream=None):
    """stem_decode_select and stem_decode_attn as one call: (out, lse, sel_idx, sel_cnt)."""
    sel_idx, sel_cnt = _lists(q, kcap, sel_idx, sel_cnt)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    _decode(_lib.stem_decode, cache, q, lens, rows, budget, kcap, method, sel_idx, sel_cnt, out,
            lse, workspace, status, stream)
    return out, lse, sel_idx, sel_cnt

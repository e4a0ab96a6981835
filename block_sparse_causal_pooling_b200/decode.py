"""Decoding with a paged K/V cache: the Python side of the decode calls in include/stem.h.

    cache = PagedCache.alloc(num_pages, Hkv, D, block, "q4", table, device)
    stem_cache_append(cache, k, v, pos)                  # K, V [nseq, Hkv, T, D] of new tokens
    budget, kcap = stem_decode_budget(cache.max_blocks, method, device)
    out, lse, sel_idx, sel_cnt = stem_decode(cache, q, lens, budget, kcap, method)

A page holds one selection block of one sequence; the caller hands pages out by writing `table`
[nseq, max_blocks]. Calls are asynchronous on `stream` (default: torch's current stream of the
cache's device) and make that device current while they launch. Tensors that a call makes itself
(outputs, workspace) are made for that stream, as under torch.cuda.stream(stream); a caller that
reads them on another stream orders the two. The calls have no gradients: outputs do not require any.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import stem as _stem
from .stem import (STEM_KV_BF16, STEM_KV_Q4, STEM_KV_Q8, STEM_SCHED_LINEAR, STEM_SHARE_GROUP,
                   STEM_SHARE_HEAD, STEM_VSUM_MAX, STEM_VSUM_MEAN, StemError, make_method,
                   stem_budget_m, stem_method_t)

try:  # (after stem: libstem.so is loaded)
    from . import _decode
except ImportError as e:
    raise ImportError("_decode.so is missing or cannot be loaded: build it with "
                      "`python -m block_sparse_causal_pooling_b200.build`") from e

_decode.set_error(StemError)
_FORMATS = {"bf16": STEM_KV_BF16, "q8": STEM_KV_Q8, "q4": STEM_KV_Q4}
_FORMAT_NAMES = {v: k for k, v in _FORMATS.items()}
_VSUMS = {"mean": STEM_VSUM_MEAN, "max": STEM_VSUM_MAX}
_VSUM_NAMES = {v: k for k, v in _VSUMS.items()}
_SHARES = {"head": STEM_SHARE_HEAD, "group": STEM_SHARE_GROUP}
_ATTN = {k: stem_method_t(share=v) for k, v in _SHARES.items()}  # all that the attention reads
_SELECT, _ATTEND = 1, 2

__all__ = ["PagedCache", "stem_cache_page_bytes", "stem_cache_append", "stem_cache_read",
           "stem_decode_budget", "stem_decode_workspace_size", "stem_decode_select",
           "stem_decode_attn", "stem_decode", "make_method", "StemError"]


def _code(table, value, name: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}") from None


def stem_cache_page_bytes(D: int, block: int, fmt: str) -> int:
    """Bytes of the record of one (page, kv head); 0 if the library does not support the shape."""
    return int(_stem.lib().stem_cache_page_bytes(D, block, _code(_FORMATS, fmt, "fmt")))


class PagedCache(_decode.Cache):
    """A paged cache over tensors that the caller owns:

    pages [num_pages, Hkv, stem_cache_page_bytes(D, block, fmt)] uint8, kbar [num_pages, Hkv, D]
    and vnorm [num_pages, Hkv] float32, table [nseq, max_blocks] int32, all contiguous on one CUDA
    device. fmt: "bf16", "q8" or "q4"; vsum: "mean" or "max" (the block summary of the V norms).
    """

    __slots__ = ()

    def __init__(self, pages, kbar, vnorm, table, block: int, fmt: str, vsum: str = "mean"):
        super().__init__(pages, kbar, vnorm, table, block, _code(_FORMATS, fmt, "fmt"),
                         _code(_VSUMS, vsum, "vsum"))

    @property
    def fmt(self) -> str:
        return _FORMAT_NAMES[self.format]

    @property
    def vsum(self) -> str:
        return _VSUM_NAMES[self.vsum_code]

    @property
    def device(self) -> torch.device:
        return self.pages.device

    @classmethod
    def alloc(cls, num_pages: int, Hkv: int, D: int, block: int, fmt: str, table: torch.Tensor,
              vsum: str = "mean") -> "PagedCache":
        """A cache with new buffers (zeroed) on the device of `table`."""
        dev = table.device
        size = stem_cache_page_bytes(D, block, fmt)
        return cls(torch.zeros((num_pages, Hkv, size), dtype=torch.uint8, device=dev),
                   torch.zeros((num_pages, Hkv, D), dtype=torch.float32, device=dev),
                   torch.zeros((num_pages, Hkv), dtype=torch.float32, device=dev), table, block,
                   fmt, vsum)


def _handle(cache: PagedCache, stream):
    """The stream's cudaStream_t; None stays None (torch's current stream of the device)."""
    if stream is None:
        return None
    if stream.device != cache.device:
        raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
    return stream.cuda_stream


# ------------------------------------------------------------------ the cache


def stem_cache_append(cache: PagedCache, k, v, pos, count=None, status=None, stream=None) -> None:
    """Write K and V rows k, v [nseq, Hkv, T, D] (bf16 or f32, any strides with a contiguous last
    dimension and rows on 16-byte boundaries) as tokens pos[s] .. pos[s] + count[s] - 1 of each
    sequence (count None: all T), quantised to the cache's format, and summarise the blocks whose
    last token is among them. A token written again in the middle of a full block leaves the block's
    summaries as they were: write on to its end to renew them."""
    _decode.append(cache, k, v, pos, count, status, _handle(cache, stream))


def stem_cache_read(cache: PagedCache, pos, count=None, k=None, v=None, T: Optional[int] = None,
                    dtype=torch.bfloat16, status=None, stream=None):
    """The values that tokens pos[s] .. pos[s] + count[s] - 1 stand for: (k, v) [nseq, Hkv, T, D],
    given, or made with T rows (rows past count then hold zeros). Rows past count of given tensors
    are left as they were."""
    if (k is None) != (v is None):
        raise ValueError("give both of k and v, or neither")
    handle = _handle(cache, stream)
    if k is None:
        if T is None:
            raise ValueError("T is needed when k and v are not given")
        with torch.cuda.stream(stream):  # (None: the current one)
            k = torch.zeros((cache.nseq, cache.Hkv, T, cache.D), dtype=dtype, device=cache.device)
            v = torch.zeros_like(k)
    _decode.read(cache, k, v, pos, count, status, handle)
    return k, v


# ------------------------------------------------------------------ decode


def stem_decode_budget(max_blocks: int, method: stem_method_t, device):
    """(budget [max_blocks] int32 on `device`, kcap): k(i) of the method's schedule for a query in
    block i, and its largest value. Made once per method and table. The linear schedule runs over a
    context's blocks, and a token is in the last block of its own: k(i) is that of the last block of
    i + 1, however wide the table is."""
    k, _ = stem_budget_m(max_blocks, method)
    if method.schedule == STEM_SCHED_LINEAR:
        k = torch.minimum(k[-1], torch.arange(1, max_blocks + 1, dtype=torch.int32))
    return k.to(device), max(int(k.max()), 1)


def stem_decode_workspace_size(cache: PagedCache, R: int, Hq: int, kcap: int) -> int:
    """Workspace bytes of a decode call of R rows; one workspace per call that may overlap another."""
    return _decode.workspace_size(cache, R, Hq, kcap)


def _method(method) -> int:
    """The address of method parameters, which the native part reads."""
    if not isinstance(method, stem_method_t):
        raise TypeError(f"method must be a stem_method_t (make_method), got {type(method).__name__}")
    return ctypes.addressof(method)


def _both(sel_idx, sel_cnt) -> None:
    if (sel_idx is None) != (sel_cnt is None):
        raise ValueError("give both of sel_idx and sel_cnt, or neither")


def stem_decode_select(cache: PagedCache, q, lens, budget, kcap: int, method: stem_method_t,
                       rows=None, sel_idx=None, sel_cnt=None, status=None, stream=None):
    """Kept blocks of query tokens q [R, Hq, D] (bf16) that see lens[r] tokens of sequence rows[r]
    (None: sequence r). Returns (sel_idx [R, Hq, kcap], ascending, -1 past the count, and sel_cnt
    [R, Hq])."""
    _both(sel_idx, sel_cnt)
    method = _method(method)
    return _decode.decode(_SELECT, cache, q, lens, rows, budget, kcap, method, sel_idx, sel_cnt,
                          None, None, None, status, _handle(cache, stream))[2:]


def stem_decode_attn(cache: PagedCache, q, lens, sel_idx, sel_cnt, share: str = "head", rows=None,
                     out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of query tokens q [R, Hq, D] over the kept blocks sel_idx [R, Hq, kcap], sel_cnt
    [R, Hq]. share "group": the query heads of a kv head have one list, that of the first. Returns
    (out [R, Hq, D] bf16, lse [R, Hq] float32)."""
    _code(_SHARES, share, "share")
    if not (isinstance(sel_idx, torch.Tensor) and isinstance(sel_cnt, torch.Tensor)):
        raise TypeError("sel_idx and sel_cnt must be tensors")
    if sel_idx.dim() != 3:
        raise ValueError(f"sel_idx must be [R, Hq, kcap], got {tuple(sel_idx.shape)}")
    return _decode.decode(_ATTEND, cache, q, lens, rows, None, sel_idx.shape[2],
                          _method(_ATTN[share]), sel_idx, sel_cnt, out, lse, workspace,
                          status, _handle(cache, stream))[:2]


def stem_decode(cache: PagedCache, q, lens, budget, kcap: int, method: stem_method_t, rows=None,
                out=None, lse=None, sel_idx=None, sel_cnt=None, workspace=None, status=None,
                stream=None):
    """stem_decode_select and stem_decode_attn as one call: (out, lse, sel_idx, sel_cnt)."""
    _both(sel_idx, sel_cnt)
    method = _method(method)
    return _decode.decode(_SELECT | _ATTEND, cache, q, lens, rows, budget, kcap, method, sel_idx,
                          sel_cnt, out, lse, workspace, status, _handle(cache, stream))

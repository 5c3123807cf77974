"""torch front end of the paged key-value cache (marshalling only).

``cache_append``, ``attn_decode`` and ``cache_evict`` run the ``bpt_cache_*``
and ``bpt_attn_decode`` calls of the library on torch tensors; include/bpt.h
defines what they compute.  A cache is four tensors that the program keeps:

  k_cache, v_cache  [pages, kv_heads, page_size, d_k], bf16 or fp16
  page_table        [B, max_pages] int32: the pages of each sequence
  lens              [B] int32: the tokens each sequence holds

and, where weights are gathered for eviction, acc (fp32) and pos (int32),
both [B, kv_heads, max_pages * page_size].  Lengths and pages stay on the
device: no call synchronises, and every call may be captured into a graph.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import _lib

_DTYPES = {torch.bfloat16: _lib.BPT_BF16, torch.float16: _lib.BPT_F16}
HEADER_BYTES = 256


def code_of(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16 or float16, got {t.dtype}")
    return code


def on_device(device: torch.device):
    """A context in which `device` is the current one (nothing if it already is)."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def new_workspace(nbytes: int, device) -> torch.Tensor:
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:HEADER_BYTES].zero_()
    return ws


def check(t: torch.Tensor, what: str, shape, dtype, device) -> int:
    """The address of a contiguous tensor of this shape, type and device."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() \
            or t.device != device:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on {device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def check_workspace(ws: torch.Tensor, device) -> torch.Tensor:
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {device}")
    return ws


def rows_check(t: torch.Tensor, what: str, shape, dtype, device) -> int:
    """The address of a tensor whose last dimension is contiguous."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device \
            or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{what} must be a {dtype} tensor {list(shape)} on {device} with its last "
                         f"dimension contiguous, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _cache(k_cache, v_cache, page_table, lens) -> "_lib.Cache":
    if k_cache.dim() != 4 or not k_cache.is_cuda or not k_cache.is_contiguous():
        raise ValueError("k_cache must be a contiguous CUDA tensor [pages, kv_heads, page_size, d_k]")
    dev = k_cache.device
    code = code_of(k_cache, "k_cache")
    pages, hkv, ps, dk = k_cache.shape
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, per = page_table.shape
    return _lib.Cache(k_cache.data_ptr(),
                      check(v_cache, "v_cache", k_cache.shape, k_cache.dtype, dev),
                      check(page_table, "page_table", page_table.shape, torch.int32, dev),
                      check(lens, "lens", (B,), torch.int32, dev),
                      B, pages, hkv, ps, dk, per, code, 0)


def _sizes(k_cache, page_table) -> "_lib.Cache":
    """The cache's sizes alone, for the workspace calls."""
    if k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, d_k], page_table "
                         "[B, max_pages]")
    pages, hkv, ps, dk = k_cache.shape
    B, per = page_table.shape
    return _lib.Cache(None, None, None, None, B, pages, hkv, ps, dk, per,
                      code_of(k_cache, "k_cache"), 0)


def cache_workspace(k_cache: torch.Tensor, page_table: torch.Tensor) -> torch.Tensor:
    """A workspace for ``cache_append`` and ``cache_evict`` on this cache."""
    st, nbytes = _lib.bpt_cache_workspace_size(_sizes(k_cache, page_table))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_cache_workspace_size")
    return new_workspace(nbytes, k_cache.device)


def attn_decode_workspace(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor,
                          with_acc: bool = False) -> torch.Tensor:
    """A workspace for ``attn_decode`` with these queries and this cache."""
    st, nbytes = _lib.bpt_attn_decode_workspace_size(_sizes(k_cache, page_table), q.shape[1],
                                                     with_acc)
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_decode_workspace_size")
    return new_workspace(nbytes, k_cache.device)


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 page_table: torch.Tensor, lens: torch.Tensor,
                 counts: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                 acc: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                 seen: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Writes the new tokens k, v [B, T, kv_heads, d_k] (any strides that are
    multiples of 8 elements, last dimension contiguous) behind each sequence;
    returns new_lens [B] (allocated if not given; not the lens tensor)."""
    c = _cache(k_cache, v_cache, page_table, lens)
    dev, B = k_cache.device, c.batch
    if k.dim() != 4:
        raise ValueError("k must be [B, T, kv_heads, d_k]")
    T = k.shape[1]
    shape = (B, T, c.kv_heads, c.d_k)
    kp = rows_check(k, "k", shape, k_cache.dtype, dev)
    vp = rows_check(v, "v", shape, k_cache.dtype, dev)
    slots = (B, c.kv_heads, c.max_pages * c.page_size)
    if new_lens is None:
        new_lens = torch.empty_like(lens)
    ws = new_workspace(HEADER_BYTES, dev) if ws is None else check_workspace(ws, dev)
    strides = (ctypes.c_int64 * 6)(*k.stride()[:3], *v.stride()[:3])
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with on_device(dev):
        st = _lib.bpt_cache_append(
            c, kp, vp, T, strides,
            None if counts is None else check(counts, "counts", (B,), torch.int32, dev),
            check(new_lens, "new_lens", (B,), torch.int32, dev),
            None if acc is None else check(acc, "acc", slots, torch.float32, dev),
            None if pos is None else check(pos, "pos", slots, torch.int32, dev),
            None if seen is None else check(seen, "seen", (B,), torch.int32, dev),
            ws.data_ptr(), ws.numel(), s.cuda_stream)
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_cache_append")
    return new_lens


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                page_table: torch.Tensor, lens: torch.Tensor, window: int = 0, sinks: int = 0,
                acc: Optional[torch.Tensor] = None, acc_out: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of one new token per sequence, q [B, heads, d_k], over the
    cache; returns out [B, heads, d_k].  With acc, the weight every slot
    received is added: acc_out = acc + weights (acc_out None: in place)."""
    c = _cache(k_cache, v_cache, page_table, lens)
    dev, B = k_cache.device, c.batch
    if q.dim() != 3:
        raise ValueError("q must be [B, heads, d_k]")
    h = q.shape[1]
    qp = rows_check(q, "q", (B, h, c.d_k), k_cache.dtype, dev)
    if out is None:
        out = torch.empty((B, h, c.d_k), dtype=q.dtype, device=dev)
    op = rows_check(out, "out", (B, h, c.d_k), k_cache.dtype, dev)
    ap = aop = None
    if acc is not None:
        slots = (B, c.kv_heads, c.max_pages * c.page_size)
        ap = check(acc, "acc", slots, torch.float32, dev)
        aop = ap if acc_out is None else check(acc_out, "acc_out", slots, torch.float32, dev)
    elif acc_out is not None:
        raise ValueError("acc_out without acc")
    ws = (attn_decode_workspace(q, k_cache, page_table, acc is not None) if ws is None
          else check_workspace(ws, dev))
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with on_device(dev):
        st = _lib.bpt_attn_decode(c, qp, h, q.stride(0), q.stride(1), window, sinks, ap, aop, op,
                                  out.stride(0), out.stride(1), ws.data_ptr(), ws.numel(),
                                  s.cuda_stream)
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_decode")
    return out


def cache_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                lens: torch.Tensor, acc: torch.Tensor, pos: torch.Tensor, seen: torch.Tensor,
                budget: int, recent: int = 0, sinks: int = 0,
                acc_out: Optional[torch.Tensor] = None, pos_out: Optional[torch.Tensor] = None,
                new_lens: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Cuts every (sequence, kv head) to at most ``budget`` slots, keeping the
    first ``sinks`` and the last ``recent`` positions and then the largest
    accumulated weights, and packs the rest; returns new_lens.  acc_out,
    pos_out, new_lens None: updated in place."""
    c = _cache(k_cache, v_cache, page_table, lens)
    dev, B = k_cache.device, c.batch
    slots = (B, c.kv_heads, c.max_pages * c.page_size)
    ap = check(acc, "acc", slots, torch.float32, dev)
    pp = check(pos, "pos", slots, torch.int32, dev)
    aop = ap if acc_out is None else check(acc_out, "acc_out", slots, torch.float32, dev)
    pop = pp if pos_out is None else check(pos_out, "pos_out", slots, torch.int32, dev)
    new_lens = lens if new_lens is None else new_lens
    ws = cache_workspace(k_cache, page_table) if ws is None else check_workspace(ws, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with on_device(dev):
        st = _lib.bpt_cache_evict(c, budget, recent, sinks, ap, pp,
                                  check(seen, "seen", (B,), torch.int32, dev), aop, pop,
                                  check(new_lens, "new_lens", (B,), torch.int32, dev),
                                  ws.data_ptr(), ws.numel(), s.cuda_stream)
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_cache_evict")
    return new_lens

"""torch front end of the paged key-value cache (marshalling only).

``cache_append``, ``attn_decode`` and ``cache_evict`` run the ``bpt_cache_*``
and ``bpt_attn_decode`` calls of the library on torch tensors; include/bpt.h
defines what they compute.  A cache is four tensors that the program keeps:

  k_cache, v_cache  [pages, kv_heads, page_size, d_k], bf16 or fp16
  page_table        [B, max_pages] int32: the pages of each sequence
  lens              [B] int32: the tokens each sequence holds

and, where weights are gathered for eviction, acc (fp32) and pos (int32),
both [B, kv_heads, max_pages * page_size].  Lengths and pages stay on the
device: no call synchronises, and every call may be captured into a graph.  With
``stream=`` a call runs with that stream current: what it allocates belongs to it.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib

_DTYPES = {torch.bfloat16: _lib.BPT_BF16, torch.float16: _lib.BPT_F16}
HEADER_BYTES = 4096  # BPT_OPS_HEADER_BYTES
_Strides = ctypes.c_int64 * 6


def code_of(t: torch.Tensor, what: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16 or float16, got {t.dtype}")
    return code


def current_stream(index: int) -> int:
    """The raw current stream of device `index`."""
    return torch._C._cuda_getCurrentRawStream(index)


def on_stream(stream: torch.cuda.Stream, t: torch.Tensor):
    """Makes `stream` current for a call on t's device: what the call allocates
    and clears is then ordered with its kernels."""
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def run(fn, index: int, *args) -> int:
    """fn(*args) with device `index` current."""
    if torch._C._cuda_getDevice() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def new_workspace(nbytes: int, device) -> torch.Tensor:
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:HEADER_BYTES].zero_()
    return ws


def _refuse(t: torch.Tensor, what: str, shape, dtype, index: int, how: str):
    raise ValueError(f"{what} must be a {dtype} tensor {list(shape)} on cuda:{index}, {how}; got "
                     f"{t.dtype} {list(t.shape)} with strides {list(t.stride())} on {t.device}")


def check(t: torch.Tensor, what: str, shape: tuple, dtype, index: int) -> int:
    """The address of a contiguous tensor of this shape and type on device `index`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index \
            or not t.is_contiguous():
        _refuse(t, what, shape, dtype, index, "contiguous")
    return t.data_ptr()


def check_workspace(ws: torch.Tensor, index: int) -> torch.Tensor:
    if ws.dtype is not torch.uint8 or ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{index}")
    return ws


def rows_check(t: torch.Tensor, what: str, shape: tuple, dtype, index: int) -> int:
    """The address of a tensor whose last dimension is contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or t.stride(-1) != 1:
        _refuse(t, what, shape, dtype, index, "its last dimension contiguous")
    return t.data_ptr()


def cache_struct(k_cache, v_cache, page_table, lens) -> "_lib.Cache":
    """The C struct of a cache, its tensors checked."""
    if k_cache.dim() != 4 or not k_cache.is_cuda or not k_cache.is_contiguous():
        raise ValueError("k_cache must be a contiguous CUDA tensor [pages, kv_heads, page_size, d_k]")
    index = k_cache.get_device()
    code = code_of(k_cache, "k_cache")
    shape = k_cache.shape
    pages, hkv, ps, dk = shape
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, per = page_table.shape
    return _lib.Cache(k_cache.data_ptr(), check(v_cache, "v_cache", shape, k_cache.dtype, index),
                      check(page_table, "page_table", (B, per), torch.int32, index),
                      check(lens, "lens", (B,), torch.int32, index),
                      B, pages, hkv, ps, dk, per, code, 0)


def cache_sizes(k_cache, page_table) -> "_lib.Cache":
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
    st, nbytes = _lib.bpt_cache_workspace_size(cache_sizes(k_cache, page_table))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_cache_workspace_size")
    return new_workspace(nbytes, k_cache.device)


def attn_decode_workspace(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor,
                          with_acc: bool = False) -> torch.Tensor:
    """A workspace for ``attn_decode`` with these queries and this cache."""
    st, nbytes = _lib.bpt_attn_decode_workspace_size(cache_sizes(k_cache, page_table), q.shape[1],
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
    if stream is not None:
        with on_stream(stream, k_cache):
            return cache_append(k, v, k_cache, v_cache, page_table, lens, counts, new_lens, acc,
                                pos, seen, ws)
    c = cache_struct(k_cache, v_cache, page_table, lens)
    index, dt, B = k_cache.get_device(), k_cache.dtype, lens.shape[0]
    if k.dim() != 4:
        raise ValueError("k must be [B, T, kv_heads, d_k]")
    _, hkv, ps, dk = k_cache.shape
    T = k.shape[1]
    shape, slots = (B, T, hkv, dk), (B, hkv, page_table.shape[1] * ps)
    kp, vp = rows_check(k, "k", shape, dt, index), rows_check(v, "v", shape, dt, index)
    if new_lens is None:
        new_lens = torch.empty_like(lens)
    ws = new_workspace(HEADER_BYTES, k_cache.device) if ws is None else check_workspace(ws, index)
    strides = _Strides(*k.stride()[:3], *v.stride()[:3])
    st = run(_lib.bpt_cache_append, index, c, kp, vp, T, strides,
             None if counts is None else check(counts, "counts", (B,), torch.int32, index),
             check(new_lens, "new_lens", (B,), torch.int32, index),
             None if acc is None else check(acc, "acc", slots, torch.float32, index),
             None if pos is None else check(pos, "pos", slots, torch.int32, index),
             None if seen is None else check(seen, "seen", (B,), torch.int32, index),
             ws.data_ptr(), ws.numel(), current_stream(index))
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
    if stream is not None:
        with on_stream(stream, k_cache):
            return attn_decode(q, k_cache, v_cache, page_table, lens, window, sinks, acc, acc_out,
                               out, ws)
    c = cache_struct(k_cache, v_cache, page_table, lens)
    index, dt, B = k_cache.get_device(), k_cache.dtype, lens.shape[0]
    if q.dim() != 3:
        raise ValueError("q must be [B, heads, d_k]")
    _, hkv, ps, dk = k_cache.shape
    h = q.shape[1]
    shape = (B, h, dk)
    qp = rows_check(q, "q", shape, dt, index)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=q.device)
    op = rows_check(out, "out", shape, dt, index)
    ap = aop = None
    if acc is not None:
        slots = (B, hkv, page_table.shape[1] * ps)
        ap = check(acc, "acc", slots, torch.float32, index)
        aop = ap if acc_out is None else check(acc_out, "acc_out", slots, torch.float32, index)
    elif acc_out is not None:
        raise ValueError("acc_out without acc")
    ws = (attn_decode_workspace(q, k_cache, page_table, acc is not None) if ws is None
          else check_workspace(ws, index))
    st = run(_lib.bpt_attn_decode, index, c, qp, h, q.stride(0), q.stride(1), window, sinks, ap,
             aop, op, out.stride(0), out.stride(1), ws.data_ptr(), ws.numel(),
             current_stream(index))
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
    if stream is not None:
        with on_stream(stream, k_cache):
            return cache_evict(k_cache, v_cache, page_table, lens, acc, pos, seen, budget, recent,
                               sinks, acc_out, pos_out, new_lens, ws)
    c = cache_struct(k_cache, v_cache, page_table, lens)
    index, B = k_cache.get_device(), lens.shape[0]
    slots = (B, k_cache.shape[1], page_table.shape[1] * k_cache.shape[2])
    ap = check(acc, "acc", slots, torch.float32, index)
    pp = check(pos, "pos", slots, torch.int32, index)
    aop = ap if acc_out is None else check(acc_out, "acc_out", slots, torch.float32, index)
    pop = pp if pos_out is None else check(pos_out, "pos_out", slots, torch.int32, index)
    new_lens = lens if new_lens is None else new_lens
    ws = cache_workspace(k_cache, page_table) if ws is None else check_workspace(ws, index)
    st = run(_lib.bpt_cache_evict, index, c, budget, recent, sinks, ap, pp,
             check(seen, "seen", (B,), torch.int32, index), aop, pop,
             check(new_lens, "new_lens", (B,), torch.int32, index), ws.data_ptr(), ws.numel(),
             current_stream(index))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_cache_evict")
    return new_lens

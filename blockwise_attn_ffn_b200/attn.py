"""torch front end of attention with a sliding window (marshalling only).

``attn_window_forward`` and ``attn_window_backward`` run the library's
``bpt_attn_window_*`` calls on torch tensors; include/bpt.h defines what they
compute.  q is [B, Nq, h, d_k], k and v
are [B, Nkv, h_kv, d_k], bf16 or fp16, with any positive strides that are
multiples of 8 elements (the parts of a packed projection as they lie).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .cache import (HEADER_BYTES, check, check_workspace, code_of, current_stream, new_workspace,
                    on_stream, rows_check, run)


def _window(q, k, window, sinks) -> "_lib.Window":
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Nq, h, d_k], k and v [B, Nkv, h_kv, d_k]")
    B, nq, h, dk = q.shape
    return _lib.Window(B, nq, k.shape[1], h, k.shape[2], dk, window, sinks, code_of(q, "q"), 0)


def _rows(t: torch.Tensor, what: str, shape: tuple, dtype, index: int) -> "_lib.Rows":
    return _lib.Rows(rows_check(t, what, shape, dtype, index), *t.stride()[:3])


def attn_window_workspace(q: torch.Tensor, k: torch.Tensor, window: int,
                          sinks: int = 0) -> torch.Tensor:
    """A workspace for ``attn_window_forward`` on tensors of these sizes."""
    st, nbytes = _lib.bpt_attn_window_workspace_size(_window(q, k, window, sinks))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_window_workspace_size")
    return new_workspace(nbytes, q.device)


def attn_window_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int,
                        sinks: int = 0, lens: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None,
                        stats: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Causal attention in which query i, at position p = Nkv - Nq + i, sees
    the keys j <= p with p - j < window or j < sinks, for rows p < lens[b]
    (others give 0); returns out [B, Nq, h, d_k].  stats: an fp32
    [B, h, Nq, 2] tensor that receives (m, l) per row, for the backward."""
    if stream is not None:
        with on_stream(stream, q):
            return attn_window_forward(q, k, v, window, sinks, lens, out, stats, ws)
    w = _window(q, k, window, sinks)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    index, dt, qs = q.get_device(), q.dtype, q.shape
    B, nq, h, dk = qs
    ks = (B, k.shape[1], k.shape[2], dk)
    if out is None:
        out = torch.empty(qs, dtype=dt, device=q.device)
    lp = None if lens is None else check(lens, "lens", (B,), torch.int32, index)
    sp = None if stats is None else check(stats, "stats", (B, h, nq, 2), torch.float32, index)
    ws = new_workspace(HEADER_BYTES, q.device) if ws is None else check_workspace(ws, index)
    st = run(_lib.bpt_attn_window_forward, index, w, _rows(q, "q", qs, dt, index),
             _rows(k, "k", ks, dt, index), _rows(v, "v", ks, dt, index), lp,
             _rows(out, "out", qs, dt, index), sp, ws.data_ptr(), ws.numel(),
             current_stream(index))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_window_forward")
    return out


def attn_window_backward_workspace(q: torch.Tensor, k: torch.Tensor, window: int,
                                   sinks: int = 0) -> torch.Tensor:
    """A workspace for ``attn_window_backward`` on tensors of these sizes."""
    st, nbytes = _lib.bpt_attn_window_backward_workspace_size(_window(q, k, window, sinks))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_window_backward_workspace_size")
    return new_workspace(nbytes, q.device)


def attn_window_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         stats: torch.Tensor, d_o: torch.Tensor, window: int, sinks: int = 0,
                         lens: Optional[torch.Tensor] = None,
                         grads: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                         ws: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None):
    """(dq, dk, dv) of ``attn_window_forward``: o and stats from it, d_o the
    gradient of o; written to grads if given (any positive strides)."""
    if stream is not None:
        with on_stream(stream, q):
            return attn_window_backward(q, k, v, o, stats, d_o, window, sinks, lens, grads, ws)
    w = _window(q, k, window, sinks)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    index, dt, qs = q.get_device(), q.dtype, q.shape
    B, nq, h, dk = qs
    ks = (B, k.shape[1], k.shape[2], dk)
    if grads is None:
        grads = (torch.empty(qs, dtype=dt, device=q.device),
                 torch.empty(ks, dtype=dt, device=q.device),
                 torch.empty(ks, dtype=dt, device=q.device))
    lp = None if lens is None else check(lens, "lens", (B,), torch.int32, index)
    if ws is None:
        ws = attn_window_backward_workspace(q, k, window, sinks)
    check_workspace(ws, index)
    st = run(_lib.bpt_attn_window_backward, index, w, _rows(q, "q", qs, dt, index),
             _rows(k, "k", ks, dt, index), _rows(v, "v", ks, dt, index),
             _rows(o, "o", qs, dt, index),
             check(stats, "stats", (B, h, nq, 2), torch.float32, index),
             _rows(d_o, "d_o", qs, dt, index), lp, _rows(grads[0], "dq", qs, dt, index),
             _rows(grads[1], "dk", ks, dt, index), _rows(grads[2], "dv", ks, dt, index),
             ws.data_ptr(), ws.numel(), current_stream(index))
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_window_backward")
    return grads

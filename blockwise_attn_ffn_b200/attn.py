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
from .cache import HEADER_BYTES, check, check_workspace, code_of, new_workspace, on_device, rows_check


def _window(q, k, window, sinks) -> "_lib.Window":
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Nq, h, d_k], k and v [B, Nkv, h_kv, d_k]")
    B, nq, h, dk = q.shape
    return _lib.Window(B, nq, k.shape[1], h, k.shape[2], dk, window, sinks, code_of(q, "q"), 0)


def _rows(t: torch.Tensor, what: str, shape, dtype, device) -> "_lib.Rows":
    p = rows_check(t, what, shape, dtype, device)
    sb, sn, sh, _ = t.stride()
    return _lib.Rows(p, sb, sn, sh)


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
    w = _window(q, k, window, sinks)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dev, dt = q.device, q.dtype
    qs, ks = (w.batch, w.n_q, w.heads, w.d_k), (w.batch, w.n_kv, w.kv_heads, w.d_k)
    if out is None:
        out = torch.empty(qs, dtype=dt, device=dev)
    rows = (_rows(q, "q", qs, dt, dev), _rows(k, "k", ks, dt, dev), _rows(v, "v", ks, dt, dev))
    lp = None if lens is None else check(lens, "lens", (w.batch,), torch.int32, dev)
    sp = None if stats is None else check(stats, "stats", (w.batch, w.heads, w.n_q, 2),
                                          torch.float32, dev)
    ws = new_workspace(HEADER_BYTES, dev) if ws is None else check_workspace(ws, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with on_device(dev):
        st = _lib.bpt_attn_window_forward(w, *rows, lp, _rows(out, "out", qs, dt, dev), sp,
                                          ws.data_ptr(), ws.numel(), s.cuda_stream)
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
    w = _window(q, k, window, sinks)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dev, dt = q.device, q.dtype
    qs, ks = (w.batch, w.n_q, w.heads, w.d_k), (w.batch, w.n_kv, w.kv_heads, w.d_k)
    if grads is None:
        grads = (torch.empty(qs, dtype=dt, device=dev), torch.empty(ks, dtype=dt, device=dev),
                 torch.empty(ks, dtype=dt, device=dev))
    lp = None if lens is None else check(lens, "lens", (w.batch,), torch.int32, dev)
    if ws is None:
        ws = attn_window_backward_workspace(q, k, window, sinks)
    check_workspace(ws, dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with on_device(dev):
        st = _lib.bpt_attn_window_backward(
            w, _rows(q, "q", qs, dt, dev), _rows(k, "k", ks, dt, dev), _rows(v, "v", ks, dt, dev),
            _rows(o, "o", qs, dt, dev),
            check(stats, "stats", (w.batch, w.heads, w.n_q, 2), torch.float32, dev),
            _rows(d_o, "d_o", qs, dt, dev), lp, _rows(grads[0], "dq", qs, dt, dev),
            _rows(grads[1], "dk", ks, dt, dev), _rows(grads[2], "dv", ks, dt, dev), ws.data_ptr(),
            ws.numel(), s.cuda_stream)
    if st != _lib.BPT_OK:
        raise _lib.BptError(st, "bpt_attn_window_backward")
    return grads

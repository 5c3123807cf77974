"""fp64 definitions of the attention operators (test infrastructure only).

``window_attention``: attention with a sliding window and sinks, by rows.
``window_attention_grads``: its gradients, from the formulas.
``decode_attention``: one token per sequence over a list of visible rows.
``evict_order``: which slots an eviction keeps and where they go.
All take and return torch float64 tensors (any device) or plain lists.
"""
from __future__ import annotations

import math
from typing import List, Optional, Tuple

import torch


def window_mask(nq: int, nkv: int, window: int, sinks: int, n: int, device) -> torch.Tensor:
    """[nq, nkv] visibility: query i stands at position p = nkv - nq + i and
    sees key j if j <= p < n and (p - j < window or j < sinks)."""
    p = torch.arange(nkv - nq, nkv, device=device)[:, None]
    j = torch.arange(nkv, device=device)[None, :]
    return (j <= p) & (p < n) & ((p - j < window) | (j < sinks))


def _heads(k: torch.Tensor, h: int) -> torch.Tensor:
    return k.repeat_interleave(h // k.shape[2], 2)


def window_attention(q, k, v, window: int, sinks: int, lens: Optional[List[int]] = None):
    """o [B, nq, h, dk], (m, l) [B, h, nq] and the weights' absolute sums
    A = sum_j p_j |v_j| (for error bounds)."""
    B, nq, h, dk = q.shape
    nkv = k.shape[1]
    kk, vv = _heads(k, h), _heads(v, h)
    o, A = torch.zeros_like(q), torch.zeros_like(q)
    m = torch.full((B, h, nq), -math.inf, dtype=q.dtype, device=q.device)
    l = torch.zeros((B, h, nq), dtype=q.dtype, device=q.device)
    for b in range(B):
        ok = window_mask(nq, nkv, window, sinks, nkv if lens is None else lens[b], q.device)
        s = torch.einsum("ihd,jhd->hij", q[b], kk[b]) / math.sqrt(dk)
        s = s.masked_fill(~ok, -math.inf)
        m[b] = s.amax(-1)
        ref = torch.where(m[b] == -math.inf, torch.zeros_like(m[b]), m[b])
        e = torch.exp(s - ref[..., None])
        l[b] = e.sum(-1)
        p = e / torch.where(l[b] == 0, torch.ones_like(l[b]), l[b])[..., None]
        # a key that a row cannot see does not count, whatever it holds
        live = ok.any(0)
        vb = torch.where(live[:, None, None], vv[b], torch.zeros_like(vv[b]))
        o[b] = torch.einsum("hij,jhd->ihd", p, vb)
        A[b] = torch.einsum("hij,jhd->ihd", p, vb.abs())
    return o, m, l, A


def window_attention_grads(q, k, v, do, window: int, sinks: int,
                           lens: Optional[List[int]] = None):
    """dq, dk, dv by dP = dO V^T, dS = P (dP - D), D = rowsum(dO * o)."""
    B, nq, h, dk_ = q.shape
    nkv, hkv = k.shape[1], k.shape[2]
    o, m, l, _ = window_attention(q, k, v, window, sinks, lens)
    kk, vv = _heads(k, h), _heads(v, h)
    dq = torch.zeros_like(q)
    gk, gv = torch.zeros_like(kk), torch.zeros_like(vv)
    sc = 1.0 / math.sqrt(dk_)
    for b in range(B):
        ok = window_mask(nq, nkv, window, sinks, nkv if lens is None else lens[b], q.device)
        row = ok.any(1)
        dob = torch.where(row[:, None, None], do[b], torch.zeros_like(do[b]))
        s = (torch.einsum("ihd,jhd->hij", q[b], kk[b]) * sc).masked_fill(~ok, -math.inf)
        ref = torch.where(m[b] == -math.inf, torch.zeros_like(m[b]), m[b])
        p = torch.exp(s - ref[..., None])
        p = p / torch.where(l[b] == 0, torch.ones_like(l[b]), l[b])[..., None]
        dp = torch.einsum("ihd,jhd->hij", dob, vv[b])
        D = torch.einsum("ihd,ihd->hi", dob, o[b])
        ds = p * (dp - D[..., None])
        dq[b] = torch.einsum("hij,jhd->ihd", ds, kk[b]) * sc
        gk[b] = torch.einsum("hij,ihd->jhd", ds, q[b]) * sc
        gv[b] = torch.einsum("hij,ihd->jhd", p, dob)
    fold = (B, nkv, hkv, h // hkv, dk_)
    return dq, gk.view(fold).sum(3), gv.view(fold).sum(3)


def visible_slots(n: int, window: int, sinks: int) -> List[int]:
    return [j for j in range(n) if window == 0 or j >= n - window or j < sinks]


def decode_attention(q, k, v) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """q [h, dk], k, v [n, hkv, dk] (the visible rows): o, p [h, n], A."""
    h, dk = q.shape
    if k.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, torch.zeros((h, 0), dtype=q.dtype, device=q.device), z
    g = h // k.shape[1]
    kk, vv = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    p = torch.softmax(torch.einsum("hd,jhd->hj", q, kk) / math.sqrt(dk), -1)
    return (torch.einsum("hj,jhd->hd", p, vv), p, torch.einsum("hj,jhd->hd", p, vv.abs()))


def evict_order(acc: List[float], pos: List[int], seen: int, budget: int, recent: int,
                sinks: int) -> List[int]:
    """For the new slots 0 .. min(n, budget) - 1, the slot that each holds
    after the eviction of one (sequence, head)."""
    n = len(acc)
    if n <= budget:
        return list(range(n))

    def rank(s):
        safe = pos[s] < sinks or pos[s] >= seen - recent
        w = acc[s]
        if safe:
            return (0, 0.0, s)
        return (2, 0.0, s) if math.isnan(w) else (1, -w, s)

    kept = sorted(sorted(range(n), key=rank)[:budget])
    keep = set(kept)
    movers = iter([s for s in kept if s >= budget])
    return [s if s in keep else next(movers) for s in range(budget)]

"""Measured cases of the windowed attention and the paged key-value cache.

Five operators, as a program that trains or serves the layer calls them:

  window_forward   attention with a sliding window and sinks (first tokens that
                   stay visible), whole sequences or a chunk behind a prefix
  window_backward  its gradients
  append           new tokens' keys and values into the pages of a cache
  decode           attention of one new token per sequence over the paged cache,
                   optionally adding up the weight that every slot received
  evict            keep the slots of largest accumulated weight, compact the rest

Each case has a plain form (elementary torch operations, fp32) and the
framework's own calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a short prompt: one sequence of a small model, latency counts
        dict(name="window_forward_short", op="window_forward", B=1, nq=200, nkv=200, h=12, hkv=12,
             dk=64, window=128, sinks=4, dtype="bf16", ragged=False, packed=True),
        # a chunk of a padded batch of prompts behind a cached prefix, shared heads
        dict(name="window_forward_chunk", op="window_forward", B=3, nq=777, nkv=1901, h=16, hkv=4,
             dk=128, window=300, sinks=64, dtype="f16", ragged=True, packed=False),
        # the long-context layer's attention under a window of 4096
        dict(name="window_forward_long", op="window_forward", B=1, nq=65536, nkv=65536, h=16,
             hkv=16, dk=128, window=4096, sinks=4, dtype="bf16", ragged=False, packed=True),
        # training step of a small model on a padded batch
        dict(name="window_backward_batch", op="window_backward", B=8, nq=2048, nkv=2048, h=12,
             hkv=12, dk=64, window=256, sinks=4, dtype="bf16", ragged=True, packed=False),
        # training step on long sequences with shared key/value heads
        dict(name="window_backward_long", op="window_backward", B=1, nq=16384, nkv=16384, h=16,
             hkv=4, dk=128, window=2048, sinks=4, dtype="f16", ragged=False, packed=False),
        # one new token of each of 64 sequences into the cache
        dict(name="append_token", op="append", B=64, T=1, hkv=8, dk=128, ps=16, top=4096,
             dtype="bf16", ragged=False, packed=True),
        # prompts of up to 8191 tokens into the cache
        dict(name="append_prompt", op="append", B=4, T=8191, hkv=16, dk=128, ps=64, top=1000,
             dtype="f16", ragged=True, packed=True),
        # one sequence, a short cache: latency counts
        dict(name="decode_one", op="decode", B=1, top=301, h=12, hkv=12, dk=64, ps=16, window=0,
             sinks=0, dtype="bf16", ragged=False, acc=False),
        # a served batch of very different lengths, shared heads, with the weights' sums
        dict(name="decode_batch", op="decode", B=64, top=8192, h=32, hkv=8, dk=128, ps=16,
             window=0, sinks=0, dtype="bf16", ragged=True, acc=True),
        # one very long sequence of the wide layer
        dict(name="decode_long", op="decode", B=1, top=131072, h=32, hkv=32, dk=128, ps=64,
             window=0, sinks=0, dtype="f16", ragged=False, acc=False),
        # a small model's caches brought back to 1024 slots
        dict(name="evict_batch", op="evict", B=8, top=1300, hkv=12, dk=64, ps=16, budget=1024,
             recent=256, sinks=4, dtype="bf16", ragged=True),
        # long caches cut to a quarter
        dict(name="evict_long", op="evict", B=4, top=65536, hkv=16, dk=128, ps=64, budget=16384,
             recent=1024, sinks=4, dtype="f16", ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_forward", "window_backward", "append", "decode", "evict"])
    dk = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    hkv = rng.choice([1, 2, 4, 8, 12, 16])
    g = rng.choice([1, 1, 2, 3, 4, 8])
    if op in ("window_forward", "window_backward"):
        top = 65536 if op == "window_forward" else 16384
        B = rng.choice([1, 1, 2, 3, 8])
        nkv = _spread(rng, 1, top // B)
        nq = nkv if rng.random() < 0.6 else _spread(rng, 1, nkv)
        h = min(hkv * g, 16) // hkv * hkv
        c = dict(op=op, B=B, nq=nq, nkv=nkv, h=h, hkv=hkv, dk=dk,
                 window=_spread(rng, 1, 3900 if op == "window_forward" else 1900),
                 sinks=rng.choice([0, 1, 4, 64, 130]), dtype=dtype, ragged=rng.random() < 0.4,
                 packed=False)
        c["packed"] = nq == nkv and h == hkv and rng.random() < 0.5
        return c
    if op == "append":
        B = _spread(rng, 1, 64)
        return dict(op=op, B=B, T=_spread(rng, 1, 32768 // B), hkv=hkv, dk=dk,
                    ps=rng.choice([16, 32, 48, 64, 128]), top=_spread(rng, 1, 4096), dtype=dtype,
                    ragged=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "decode":
        B = _spread(rng, 1, 64)
        window = rng.choice([0, 0, _spread(rng, 1, 8192)])
        return dict(op=op, B=B, top=_spread(rng, 1, 250000 // B), h=hkv * g, hkv=hkv, dk=dk,
                    ps=rng.choice([16, 32, 48, 64, 128]), window=window,
                    sinks=rng.choice([1, 4, 70]) if window else 0, dtype=dtype,
                    ragged=rng.random() < 0.5, acc=rng.random() < 0.5)
    B = _spread(rng, 1, 16)
    top = _spread(rng, 16, 262144 // B)
    budget = _spread(rng, 8, top)
    return dict(op=op, B=B, top=top, hkv=hkv, dk=dk, ps=rng.choice([16, 32, 48, 64, 128]),
                budget=budget, recent=rng.randint(0, budget // 2),
                sinks=rng.choice([0, 1, 4]), dtype=dtype, ragged=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs --
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _lengths(g, B, top, ragged, low=None):
    """Lengths on the device: all `top`, or spread over low..top with one of `top`."""
    if not ragged:
        return torch.full((B,), top, dtype=torch.int32, device="cuda")
    low = max(1, top // 4) if low is None else low
    n = torch.randint(low, top + 1, (B,), generator=g, device="cuda", dtype=torch.int64)
    n[B // 2] = top
    return n.to(torch.int32)


def _pages(g, B, slots, ps):
    """A page table whose pages lie in any order in a pool with some pages to spare."""
    per = -(-slots // ps)
    total = B * per + 3
    order = torch.randperm(total, generator=g, device="cuda")[:B * per]
    return order.view(B, per).to(torch.int32).contiguous(), total


def prepare(case, seed):
    c, g = case, _generator(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("window_forward", "window_backward"):
        B, nq, nkv, h, hkv, dk = (c[k] for k in ("B", "nq", "nkv", "h", "hkv", "dk"))
        if c["packed"]:  # the three parts of one projection
            qkv = _normal(g, (B, nkv, 3, h, dk), dt)
            s["q"], s["k"], s["v"] = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
        else:
            s["q"] = _normal(g, (B, nq, h, dk), dt)
            s["k"] = _normal(g, (B, nkv, hkv, dk), dt)
            s["v"] = _normal(g, (B, nkv, hkv, dk), dt)
        s["lens"] = _lengths(g, B, nkv, True) if c["ragged"] else None
        if c["op"] == "window_forward":
            s["out"] = torch.empty((B, nq, h, dk), dtype=dt, device="cuda")
        else:
            o, m, l = _plain_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"], s["lens"])
            s["o"], s["stats"] = o.to(dt), torch.stack([m, l], dim=-1).contiguous()
            s["do"] = _normal(g, (B, nq, h, dk), dt)
            s["grads"] = tuple(torch.empty_like(s[k], memory_format=torch.contiguous_format)
                               for k in ("q", "k", "v"))
        if own:
            import blockwise_attn_ffn_b200 as bpt
            make = (bpt.attn_window_workspace if c["op"] == "window_forward"
                    else bpt.attn_window_backward_workspace)
            s["ws"] = make(s["q"], s["k"], c["window"], c["sinks"])
        return s
    B, hkv, dk, ps = c["B"], c["hkv"], c["dk"], c["ps"]
    slots = c["top"] + (c["T"] if c["op"] == "append" else 0)
    s["table"], total = _pages(g, B, slots, ps)
    S = s["table"].shape[1] * ps
    s["kc"] = _normal(g, (total, hkv, ps, dk), dt)
    s["vc"] = _normal(g, (total, hkv, ps, dk), dt)
    s["lens"] = _lengths(g, B, c["top"], c["ragged"])
    if c["op"] == "append":
        T = c["T"]
        if c["packed"]:
            kv = _normal(g, (B, T, 2, hkv, dk), dt)
            s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        else:
            s["k"], s["v"] = _normal(g, (B, T, hkv, dk), dt), _normal(g, (B, T, hkv, dk), dt)
        s["counts"] = _lengths(g, B, T, True, 0) if c["ragged"] else None
        s["acc"] = torch.rand((B, hkv, S), generator=g, device="cuda")
        s["pos"] = torch.arange(S, device="cuda", dtype=torch.int32).repeat(B, hkv, 1)
        s["seen"] = s["lens"] + 7
        s["new_lens"] = torch.zeros_like(s["lens"])
    elif c["op"] == "decode":
        s["q"] = _normal(g, (B, c["h"], dk), dt, 1.5)
        s["out"] = torch.empty((B, c["h"], dk), dtype=dt, device="cuda")
        s["acc"] = s["acc_out"] = None
        if c["acc"]:
            s["acc"] = torch.rand((B, hkv, S), generator=g, device="cuda") * 0.01
            s["acc_out"] = s["acc"].clone()
    else:
        # weights gathered over many steps: a few slots hold most, some none at all
        a = torch.randn((B, hkv, S), generator=g, device="cuda").mul(2.0).exp()
        s["acc"] = torch.where(torch.rand((B, hkv, S), generator=g, device="cuda") < 0.1,
                               torch.zeros_like(a), a)
        # an earlier eviction left gaps in the positions, in any order of the slots
        s["pos"] = (torch.rand((B, hkv, S), generator=g, device="cuda").argsort(-1) * 2).to(
            torch.int32)
        s["seen"] = torch.full((B,), 2 * S, dtype=torch.int32, device="cuda")
        s["acc_out"], s["pos_out"] = torch.zeros_like(s["acc"]), torch.zeros_like(s["pos"])
        s["new_lens"] = torch.zeros_like(s["lens"])
    if own:
        import blockwise_attn_ffn_b200 as bpt
        if c["op"] == "append":
            s["ws"] = bpt.cache_workspace(s["kc"], s["table"])
        elif c["op"] == "decode":
            s["ws"] = bpt.attn_decode_workspace(s["q"], s["kc"], s["table"], c["acc"])
        else:
            s["ws"] = bpt.cache_workspace(s["kc"], s["table"])
    return s


# ------------------------------------------------------------- plain forms --
def _seen_keys(p0, p1, window, sinks):
    """The key range and the number of sink keys before it that queries p0..p1-1 can see."""
    lo = max(0, p0 - window + 1)
    return lo, min(sinks, lo)


def _plain_chunks(q, k, v, window, sinks, lens, rows=1024):
    """Per sequence and chunk of queries: fp32 tensors by key/value head and the mask."""
    B, nq, h, dk = q.shape
    nkv, hkv = k.shape[1], k.shape[2]
    for b in range(B):
        n = nkv if lens is None else lens[b]
        for i0 in range(0, nq, rows):
            i1 = min(nq, i0 + rows)
            p0, p1 = nkv - nq + i0, nkv - nq + i1
            lo, ns = _seen_keys(p0, p1, window, sinks)
            j = torch.cat([torch.arange(ns, device=q.device),
                           torch.arange(lo, p1, device=q.device)])
            p = torch.arange(p0, p1, device=q.device)[:, None]
            mask = (j <= p) & ((p - j < window) | (j < sinks)) & (p < n)
            qc = q[b, i0:i1].float().permute(1, 0, 2).reshape(hkv, h // hkv, i1 - i0, dk)
            kc = torch.cat([k[b, :ns], k[b, lo:p1]]).float().permute(1, 0, 2)[:, None]
            vc = torch.cat([v[b, :ns], v[b, lo:p1]]).float().permute(1, 0, 2)[:, None]
            yield b, i0, i1, j, mask, qc, kc, vc


def _plain_forward(q, k, v, window, sinks, lens):
    B, nq, h, dk = q.shape
    o = torch.empty((B, nq, h, dk), dtype=torch.float32, device=q.device)
    m = torch.empty((B, h, nq), dtype=torch.float32, device=q.device)
    l = torch.empty_like(m)
    for b, i0, i1, j, mask, qc, kc, vc in _plain_chunks(q, k, v, window, sinks, lens):
        x = torch.matmul(qc, kc.transpose(-1, -2)).mul_(1.0 / math.sqrt(dk))
        x.masked_fill_(~mask, -math.inf)
        mx = x.amax(-1, keepdim=True)
        x.sub_(torch.where(mx == -math.inf, torch.zeros_like(mx), mx)).exp_()
        sm = x.sum(-1, keepdim=True)
        y = torch.matmul(x, vc) / torch.where(sm == 0, torch.ones_like(sm), sm)
        o[b, i0:i1] = y.reshape(h, i1 - i0, dk).permute(1, 0, 2)
        m[b, :, i0:i1] = mx.reshape(h, i1 - i0)
        l[b, :, i0:i1] = sm.reshape(h, i1 - i0)
    return o, m, l


def _plain_backward(s):
    c = s["case"]
    q, k, v = s["q"], s["k"], s["v"]
    B, nq, h, dk = q.shape
    hkv = k.shape[2]
    dq = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    dk_ = torch.zeros(k.shape, dtype=torch.float32, device=q.device)
    dv_ = torch.zeros(v.shape, dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(dk)
    for b, i0, i1, j, mask, qc, kc, vc in _plain_chunks(q, k, v, c["window"], c["sinks"],
                                                        s["lens"]):
        n, shape = i1 - i0, (hkv, h // hkv, i1 - i0)
        m = s["stats"][b, :, i0:i1, 0].reshape(*shape, 1)
        l = s["stats"][b, :, i0:i1, 1].reshape(*shape, 1)
        p = torch.matmul(qc, kc.transpose(-1, -2)).mul_(sc)
        p = p.sub_(torch.where(l == 0, torch.zeros_like(m), m)).masked_fill_(~mask, -math.inf)
        p = p.exp_().div_(torch.where(l == 0, torch.ones_like(l), l))
        do = s["do"][b, i0:i1].float().permute(1, 0, 2).reshape(*shape, dk)
        o = s["o"][b, i0:i1].float().permute(1, 0, 2).reshape(*shape, dk)
        ds = torch.matmul(do, vc.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        dq[b, i0:i1] = (torch.matmul(ds, kc) * sc).reshape(h, n, dk).permute(1, 0, 2)
        a = (torch.matmul(ds.transpose(-1, -2), qc) * sc).sum(1).permute(1, 0, 2)
        w = torch.matmul(p.transpose(-1, -2), do).sum(1).permute(1, 0, 2)
        dk_[b].index_add_(0, j, a)
        dv_[b].index_add_(0, j, w)
    return tuple(x.to(q.dtype) for x in (dq, dk_, dv_))


def _plain_append(s):
    c = s["case"]
    T, ps = c["T"], c["ps"]
    lens = s["lens"].long()
    counts = torch.full_like(lens, T) if s["counts"] is None else s["counts"].long()
    b, t = torch.nonzero(torch.arange(T, device=lens.device) < counts[:, None], as_tuple=True)
    slot = lens[b] + t
    page = s["table"][b, slot // ps].long()
    s["kc"][page, :, slot % ps] = s["k"][b, t]
    s["vc"][page, :, slot % ps] = s["v"][b, t]
    s["acc"][b, :, slot] = 0.0
    s["pos"][b, :, slot] = (s["seen"].long()[b] + t).to(torch.int32)[:, None]
    s["new_lens"].copy_(lens + counts)
    return s["kc"], s["vc"], s["acc"], s["pos"], s["new_lens"]


def _gathered(cache, table, b):
    """A sequence's rows in slot order, fp32 [hkv, slots, dk]."""
    x = cache[table[b].long()].float()
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])


def _plain_decode(s):
    c = s["case"]
    q, hkv = s["q"], c["hkv"]
    B, h, dk = q.shape
    out = torch.empty((B, h, dk), dtype=torch.float32, device=q.device)
    for b in range(B):
        k, v = _gathered(s["kc"], s["table"], b), _gathered(s["vc"], s["table"], b)
        slot = torch.arange(k.shape[1], device=q.device)
        live = slot < s["lens"][b]
        mask = live
        if c["window"]:
            mask = live & ((slot >= s["lens"][b] - c["window"]) | (slot < c["sinks"]))
        x = torch.matmul(q[b].float().view(hkv, h // hkv, dk), k.transpose(-1, -2))
        x = (x / math.sqrt(dk)).masked_fill(~mask, -math.inf)
        x = (x - x.amax(-1, keepdim=True)).exp()
        x = x / x.sum(-1, keepdim=True)
        out[b] = torch.matmul(x, v).reshape(h, dk)
        if s["acc"] is not None:
            s["acc_out"][b] = torch.where(live, s["acc"][b] + x.sum(1), s["acc_out"][b])
    out = out.to(q.dtype)
    return (out,) if s["acc"] is None else (out, s["acc_out"])


def _plain_evict(s):
    c = s["case"]
    acc, pos, ps, budget = s["acc"], s["pos"], c["ps"], c["budget"]
    slot = torch.arange(acc.shape[2], device=acc.device)
    lens = s["lens"].long()[:, None, None]
    live = slot < lens
    safe = (pos < c["sinks"]) | (pos >= (s["seen"][:, None, None] - c["recent"]))
    # by weight from the largest, equal ones by slot: a stable sort
    key = torch.where(safe, torch.full_like(acc, math.inf), acc)
    key = torch.where(live, key, torch.full_like(acc, -math.inf))
    order = key.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order).contiguous())
    kept = live & (rank < budget)
    new = lens.clamp(max=budget)
    s["acc_out"].copy_(torch.where(kept & (slot < new), acc, s["acc_out"]))
    s["pos_out"].copy_(torch.where(kept & (slot < new), pos, s["pos_out"]))
    hb, hh, hole = torch.nonzero(live & ~kept & (slot < new), as_tuple=True)
    mb, mh, mover = torch.nonzero(kept & (slot >= new), as_tuple=True)
    s["acc_out"][hb, hh, hole] = acc[mb, mh, mover]
    s["pos_out"][hb, hh, hole] = pos[mb, mh, mover]
    to, fro = s["table"][hb, hole // ps].long(), s["table"][mb, mover // ps].long()
    for x in (s["kc"], s["vc"]):
        x[to, hh, hole % ps] = x[fro, mh, mover % ps]
    s["new_lens"].copy_(new.view(-1))
    return s["kc"], s["vc"], s["acc_out"], s["pos_out"], s["new_lens"]


# -------------------------------------------------------------------- run --
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "window_forward":
            return _plain_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"],
                                  s["lens"])[0].to(s["q"].dtype)
        return {"window_backward": _plain_backward, "append": _plain_append,
                "decode": _plain_decode, "evict": _plain_evict}[op](s)
    import blockwise_attn_ffn_b200 as bpt
    if op == "window_forward":
        return bpt.attn_window_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"],
                                       lens=s["lens"], out=s["out"], ws=s["ws"])
    if op == "window_backward":
        return bpt.attn_window_backward(s["q"], s["k"], s["v"], s["o"], s["stats"], s["do"],
                                        c["window"], c["sinks"], lens=s["lens"],
                                        grads=s["grads"], ws=s["ws"])
    if op == "append":
        bpt.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                         counts=s["counts"], new_lens=s["new_lens"], acc=s["acc"], pos=s["pos"],
                         seen=s["seen"], ws=s["ws"])
        return s["kc"], s["vc"], s["acc"], s["pos"], s["new_lens"]
    if op == "decode":
        o = bpt.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=c["window"],
                            sinks=c["sinks"], acc=s["acc"], acc_out=s["acc_out"], out=s["out"],
                            ws=s["ws"])
        return (o,) if s["acc"] is None else (o, s["acc_out"])
    bpt.cache_evict(s["kc"], s["vc"], s["table"], s["lens"], s["acc"], s["pos"], s["seen"],
                    c["budget"], c["recent"], c["sinks"], acc_out=s["acc_out"],
                    pos_out=s["pos_out"], new_lens=s["new_lens"], ws=s["ws"])
    return s["kc"], s["vc"], s["acc_out"], s["pos_out"], s["new_lens"]


# ------------------------------------------------------------------- work --
def _visible_pairs(c, n):
    """Visible (query, key) pairs of one sequence of n valid keys."""
    w, k, off = c["window"], c["sinks"], c["nkv"] - c["nq"]
    total = 0
    for p in range(off, min(n, c["nkv"])):
        lo = max(0, p - w + 1)
        total += p + 1 - lo + min(k, lo)
    return total


def work(case):
    c = case
    if c["op"] in ("window_forward", "window_backward"):
        # a ragged batch has about 5/8 of the full lengths
        n = c["nkv"] * 5 // 8 if c["ragged"] else c["nkv"]
        off = c["nkv"] - c["nq"]
        pairs = c["B"] * c["h"] * _visible_pairs(c, n)
        rows = c["B"] * max(0, n - off)
        keys = c["B"] * n
        qb, kb = rows * c["h"] * c["dk"] * 2, keys * c["hkv"] * c["dk"] * 2
        if c["op"] == "window_forward":
            return {"bytes": 2 * qb + 2 * kb, "flops": 4 * c["dk"] * pairs}
        return {"bytes": 4 * qb + 4 * kb + rows * c["h"] * 8, "flops": 10 * c["dk"] * pairs}
    part = 5 / 8 if c["ragged"] else 1.0
    row = c["hkv"] * c["dk"] * 2
    if c["op"] == "append":
        n = c["B"] * c["T"] * (0.5 if c["ragged"] else 1.0)
        return {"bytes": int(n * (4 * row + 8 * c["hkv"])), "flops": 0}
    n = c["top"] * part
    if c["op"] == "decode":
        seen = min(n, c["window"] + c["sinks"]) if c["window"] else n
        return {"bytes": int(c["B"] * (2 * seen * row + (8 * n * c["hkv"] if c["acc"] else 0) +
                                       4 * c["h"] * c["dk"])),
                "flops": int(4 * c["B"] * c["h"] * c["dk"] * seen)}
    gone = max(0.0, n - c["budget"])
    moved = gone * min(1.0, c["budget"] / max(n, 1))  # of the evicted, those before the budget
    return {"bytes": int(c["B"] * c["hkv"] * (8 * n + 8 * min(n, c["budget"]) +
                                              moved * 4 * c["dk"] * 2)),
            "flops": 0}


# ------------------------------------------------- the definition, 64 bits --
def _exact_rows(q, k, v, first, window, sinks, n):
    """Attention of the queries q [r, h, dk] at positions first.. over every key that one of
    them can see, from the definition: h heads of q, hkv of k and v."""
    r, h, dk = q.shape
    g = h // k.shape[1]
    pos = first + torch.arange(r, device=q.device)
    key = torch.arange(k.shape[0], device=q.device)
    near = (key > first - window) & (key < first + r)
    use = key[near | ((key < sinks) & (key < first + r))]
    gap = pos[:, None] - use[None, :]
    ok = (gap >= 0) & ((gap < window) | (use < sinks)[None, :])
    score = torch.einsum("ihd,jhd->hij", q, k[use].repeat_interleave(g, 1)) / dk ** 0.5
    weight = torch.softmax(score.masked_fill(~ok, float("-inf")), -1)
    out = torch.einsum("hij,jhd->ihd", weight, v[use].repeat_interleave(g, 1))
    return torch.where((pos < n)[:, None, None], out, torch.zeros_like(out))


def exact(case, seed):
    c = case
    if c["op"] == "append":
        return None  # values that are copied: compared as they are
    s = prepare(case, seed)
    if c["op"] in ("window_forward", "window_backward"):
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        lens = [c["nkv"]] * c["B"] if s["lens"] is None else s["lens"].tolist()
        off, step = c["nkv"] - c["nq"], 512
        if c["op"] == "window_forward":
            out = torch.zeros_like(q)
            for b in range(c["B"]):
                for i in range(0, c["nq"], step):
                    out[b, i:i + step] = _exact_rows(q[b, i:i + step], k[b], v[b], off + i,
                                                     c["window"], c["sinks"], lens[b])
            return out
        dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b in range(c["B"]):
            for i in range(0, c["nq"], step):
                leaves = [x.detach().clone().requires_grad_() for x in (q[b, i:i + step], k[b],
                                                                        v[b])]
                o = _exact_rows(*leaves, off + i, c["window"], c["sinks"], lens[b])
                got = torch.autograd.grad(o, leaves, s["do"][b, i:i + step].double())
                dq[b, i:i + step] = got[0]
                dk_[b] += got[1]
                dv_[b] += got[2]
        return dq, dk_, dv_
    if c["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        acc = None if s["acc"] is None else s["acc_out"].double()
        g = c["h"] // c["hkv"]
        for b, n in enumerate(s["lens"].tolist()):
            slot = torch.arange(n, device="cuda")
            if c["window"]:
                slot = slot[(slot < c["sinks"]) | (n - slot <= c["window"])]
            page = s["table"][b].long()[slot // c["ps"]]
            if acc is not None:
                acc[b, :, :n] = s["acc"][b, :, :n].double()
            for t in range(c["hkv"]):
                k = s["kc"][page, t, slot % c["ps"]].double()
                v = s["vc"][page, t, slot % c["ps"]].double()
                p = torch.softmax(s["q"][b, t * g:(t + 1) * g].double() @ k.T / c["dk"] ** 0.5, -1)
                out[b, t * g:(t + 1) * g] = p @ v
                if acc is not None:
                    acc[b, t, slot] += p.sum(0)
        return (out,) if acc is None else (out, acc)
    # eviction: the state beside the cache's rows, one head at a time on the host
    acc, pos = s["acc"].double().cpu().numpy(), s["pos"].cpu().numpy()
    a_out, p_out = s["acc_out"].double().cpu(), s["pos_out"].cpu()
    new = []
    for b, n in enumerate(s["lens"].tolist()):
        new.append(min(n, c["budget"]))
        recent = s["seen"][b].item() - c["recent"]
        for t in range(c["hkv"]):
            w, at = acc[b, t, :n], pos[b, t, :n]
            free = (at >= c["sinks"]) & (at < recent)
            keep = np.sort(np.lexsort((np.arange(n), -w, free))[:new[b]])
            fro = np.arange(new[b])
            fro[~np.isin(fro, keep)] = keep[keep >= new[b]]
            a_out[b, t, :new[b]] = torch.from_numpy(w[fro])
            p_out[b, t, :new[b]] = torch.from_numpy(at[fro])
    return None, None, a_out, p_out, torch.tensor(new, dtype=torch.int32)

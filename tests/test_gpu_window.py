"""Attention with a sliding window and sinks on the GPU against its fp64
definition (oracle/attention.py)."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import window_attention, window_mask

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)


def no_fault(ws):
    st, site = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_OK, (bpt.status_string(st), site)


def inputs(seed, B, nq, nkv, h, hkv, dk, dt, packed=False, scale=1.0):
    g = gen(seed)
    if packed:
        qkv = randn(g, (B, nkv, 3, h, dk), dt, scale)
        return qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    return (randn(g, (B, nq, h, dk), dt, scale), randn(g, (B, nkv, hkv, dk), dt, scale),
            randn(g, (B, nkv, hkv, dk), dt))


def score_error(q, k):
    """Bound of the error of s = q.k / sqrt(dk) in fp32: 2 dk 2^-24 of the sum
    of the products' magnitudes (also where the tensor core truncates)."""
    dk = q.shape[-1]
    m = q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()
    return 2 * dk * 2.0 ** -24 * m.item() / math.sqrt(dk)


def bounds(q, k, dt, n):
    """(u, c): half a step of the type; the relative error of a weight in fp32
    (its own score's and the sum's, exp2 by the unit 2^-21 or by the cubic
    7.6e-5, sums over n keys)."""
    return torch.finfo(dt).eps / 2, 2 * score_error(q, k) + 2 * 7.6e-5 + n * 2.0 ** -23


CASES = [
    # B, nq, nkv, h, hkv, dk, window, sinks, dtype, lens, packed
    (1, 1, 1, 1, 1, 64, 1, 0, "bf16", None, False),
    (2, 1, 300, 4, 2, 128, 100, 4, "f16", None, False),
    (1, 200, 200, 2, 2, 64, 128, 4, "bf16", None, True),
    (1, 513, 513, 3, 1, 128, 1, 0, "f16", None, False),
    (1, 640, 640, 2, 1, 64, 1, 130, "bf16", None, False),
    (3, 77, 301, 6, 2, 128, 60, 64, "bf16", [301, 250, 10], False),
    (2, 257, 257, 5, 5, 64, 300, 0, "f16", [257, 0], True),
    (2, 384, 384, 4, 1, 128, 127, 1, "bf16", [129, 128], False),
    (1, 1000, 1901, 2, 2, 128, 300, 300, "f16", None, False),
    (1, 1537, 1537, 2, 1, 64, 5000, 0, "bf16", [1400], False),   # plain causal
    (1, 2048, 2048, 1, 1, 128, 256, 4, "bf16", None, True),
    (1, 512, 512, 1, 1, 64, 255, 200, "bf16", None, False),      # sinks across the window's start
    (1, 129, 4000, 3, 3, 64, 1999, 130, "f16", [3950], False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:9])))
def test_window_forward_against_the_definition(case):
    B, nq, nkv, h, hkv, dk, window, sinks, dt, lens, packed = case
    dt = DT[dt]
    q, k, v = inputs(1, B, nq, nkv, h, hkv, dk, dt, packed)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = bpt.attn_window_workspace(q, k, window, sinks)
    out = torch.full((B, nq, h, dk), math.nan, dtype=dt, device="cuda")
    stats = torch.full((B, h, nq, 2), math.nan, device="cuda")
    got = bpt.attn_window_forward(q, k, v, window, sinks, lens=lt, out=out, stats=stats, ws=ws)
    assert got is out
    no_fault(ws)
    o, m, l, A = window_attention(q.double(), k.double(), v.double(), window, sinks, lens)
    u, c = bounds(q, k, dt, min(nkv, window + sinks))
    err = (out.double() - o).abs()
    # weights rounded once (and by fp32's error), the result once; fp16 weights
    # below 2^-14 of the reference are off by 2^-25 of it at most
    tiny = 2.0 ** -25 * min(nkv, window + sinks) * v.abs().max().item() if dt == torch.float16 else 0
    tol = (u + c) * A * (1 + u) + u * o.abs() + 2.0 ** -25 + tiny
    assert (err <= tol).all(), (err - tol).max().item()
    dead = m == -math.inf
    assert (stats[..., 0][dead] == -math.inf).all() and (stats[..., 1][dead] == 0).all()
    s_err = score_error(q, k) + 2.0 ** -22 * (1 + m[~dead].abs())
    assert ((stats[..., 0] - m).abs()[~dead] <= (s_err if s_err.numel() else 1)).all()
    # l from the stored m: exp of the difference of the two maxima is part of it
    rel = (stats[..., 1].double() * torch.exp(stats[..., 0].double() - m) / l - 1).abs()[~dead]
    assert (rel <= c + 2.0 ** -20).all(), rel.max().item()
    if lens is not None:
        for b in range(B):
            first = max(0, lens[b] - (nkv - nq))
            assert (out[b, first:] == 0).all()


def test_rows_are_the_dense_softmax_of_one_key():
    """A window of one key: the output is that key's value, exactly."""
    q, k, v = inputs(2, 2, 400, 400, 4, 2, 64, torch.bfloat16)
    out = bpt.attn_window_forward(q, k, v, 1)
    assert torch.equal(out, v.repeat_interleave(2, 2))


@pytest.mark.parametrize("dt,dk", [("bf16", 64), ("f16", 128)])
def test_masked_nan_and_infinity_do_not_reach_a_row(dt, dk):
    """NaN and infinities in padding, past the window and in the future change
    only the rows that see them."""
    dt = DT[dt]
    B, n, h, hkv, window, sinks = 2, 600, 4, 2, 100, 3
    lens = [600, 333]
    q, k, v = inputs(3, B, n, n, h, hkv, dk, dt)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = bpt.attn_window_forward(q, k, v, window, sinks, lens=lt)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    bad = {(0, 50): (math.nan, math.inf), (0, 301): (1.0, math.nan), (0, 599): (math.inf, 1.0),
           (1, 200): (1.0, -math.inf)}
    for (b, j), (kx, vx) in bad.items():
        k2[b, j], v2[b, j] = kx, vx
    for x in (q2, k2, v2):
        x[1, 333:] = math.nan
    out = bpt.attn_window_forward(q2, k2, v2, window, sinks, lens=lt)
    for b in range(B):
        mask = window_mask(n, n, window, sinks, lens[b], "cuda")
        hit = torch.zeros(n, dtype=torch.bool, device="cuda")
        for (bb, j) in bad:
            if bb == b:
                hit |= mask[:, j]
        same = ~hit
        # rows past their window of a planted key are done again in fp32:
        # as near to the clean ones as two roundings of P and o allow
        a, c = out[b][same].double(), clean[b][same].double()
        assert torch.isfinite(a).all()
        u = torch.finfo(dt).eps / 2
        A = window_attention(q[b:b + 1].double(), k[b:b + 1].double(), v[b:b + 1].double(), window,
                             sinks, lens[b:b + 1])[3][0][same]
        assert ((a - c).abs() <= 2.1 * u * (A + c.abs()) + 4e-4 * A + 2.0 ** -24).all()
        assert not torch.isfinite(out[b][hit]).all(-1).any()


def test_strides_streams_devices_and_graphs():
    """Rows in wider buffers, heads before tokens, another stream, a captured
    and replayed call: bitwise what the plain call gives."""
    B, n, h, hkv, dk = 2, 300, 4, 2, 64
    q, k, v = inputs(4, B, n, n, h, hkv, dk, torch.float16)
    want = bpt.attn_window_forward(q, k, v, 90, 5)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)          # [B, h, N, dk] in memory
    kw = torch.zeros(B, n, hkv, dk + 24, dtype=q.dtype, device="cuda")[..., :dk].copy_(k)
    vw = torch.zeros(n, B, hkv, dk, dtype=q.dtype, device="cuda").transpose(0, 1).copy_(v)
    wide = torch.full((B, n, h, dk + 8), 7.0, dtype=q.dtype, device="cuda")
    ws = bpt.attn_window_workspace(q, k, 90, 5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bpt.attn_window_forward(qt, kw, vw, 90, 5, out=wide[..., :dk], ws=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(wide[..., :dk], want) and (wide[..., dk:] == 7.0).all()
    lens = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bpt.attn_window_forward(q, k, v, 90, 5, lens=lens, out=out, ws=ws)
    graph.replay()
    assert torch.equal(out, want)
    lens.copy_(torch.tensor([0, 171], dtype=torch.int32))
    graph.replay()
    assert (out[0] == 0).all() and (out[1, 171:] == 0).all()
    assert torch.equal(out[1, :171], bpt.attn_window_forward(q, k, v, 90, 5, lens=lens)[1, :171])
    no_fault(ws)


def test_a_length_outside_the_keys_is_reported():
    q, k, v = inputs(5, 2, 100, 100, 2, 2, 64, torch.bfloat16)
    lens = torch.tensor([-3, 1000], dtype=torch.int32, device="cuda")
    ws = bpt.attn_window_workspace(q, k, 50)
    out = bpt.attn_window_forward(q, k, v, 50, lens=lens, ws=ws)
    st, site = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_ERR_INDEX and site != 0
    assert (out[0] == 0).all()
    assert torch.equal(out[1], bpt.attn_window_forward(q, k, v, 50)[1])


def test_chunks_give_the_rows_of_the_whole():
    """Chunks of queries behind their prefix: the same rows as the whole
    sequence at once (other tiles, so up to the roundings)."""
    n, h, hkv, dk, window, sinks = 900, 4, 2, 128, 200, 8
    q, k, v = inputs(6, 1, n, n, h, hkv, dk, torch.bfloat16)
    whole = bpt.attn_window_forward(q, k, v, window, sinks)
    A = window_attention(q.double(), k.double(), v.double(), window, sinks)[3]
    u = torch.finfo(q.dtype).eps / 2
    at = 0
    for size in (1, 130, 269, 500):
        end = at + size
        got = bpt.attn_window_forward(q[:, at:end], k[:, :end], v[:, :end], window, sinks)
        d = (got.double() - whole[:, at:end].double()).abs()
        assert (d <= 2.1 * u * (A[:, at:end] + whole[:, at:end].double().abs()) + 4e-4 * A[:, at:end]).all()
        at = end

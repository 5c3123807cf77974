"""Gradients of attention with a sliding window on the GPU against the fp64
formulas (oracle/attention.py) and against differences of the forward."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import window_attention, window_attention_grads, window_mask
from test_gpu_window import DT, gen, inputs, no_fault, randn, score_error

pytestmark = pytest.mark.gpu


def forward(q, k, v, window, sinks, lens):
    stats = torch.empty((q.shape[0], q.shape[2], q.shape[1], 2), device="cuda")
    o = bpt.attn_window_forward(q, k, v, window, sinks, lens=lens, stats=stats)
    return o, stats


def grad_bounds(q, k, v, o, do, window, sinks, lens):
    """Elementwise bounds of the kernels' gradients, from what is rounded: P
    once (u), dS once more (u), the results once (u); o, which enters D, was
    rounded by the forward (u |dO| |o| per row); fp32 leaves c in the weights
    and e in dP (as for scores); sums over n terms add n 2^-23.  fp16: P below
    2^-22 and dS below 2^-18 of the largest |dO| are in the subnormals, off by
    2^-33 and 2^-29 max |dO| at most (scaled by 2^8, and 2^4 over max |dO|)."""
    dt = q.dtype
    u = torch.finfo(dt).eps / 2
    B, nq, h, dk = q.shape
    nkv, hkv = k.shape[1], k.shape[2]
    g = h // hkv
    c = 2 * score_error(q, k) + 2 * 7.6e-5 + min(nkv, window + sinks) * 2.0 ** -23
    sc = 1 / math.sqrt(dk)
    Q, O, DO = q.double(), o.double(), do.double()
    K, V = k.double().repeat_interleave(g, 2), v.double().repeat_interleave(g, 2)
    bq, bk, bv = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(K)
    n = [nkv] * B if lens is None else lens
    for b in range(B):
        ok = window_mask(nq, nkv, window, sinks, n[b], "cuda")
        row = ok.any(1)
        D_o = torch.where(row[:, None, None], DO[b], torch.zeros_like(DO[b]))
        Qb = torch.where(row[:, None, None], Q[b], torch.zeros_like(Q[b]))
        col = ok.any(0)
        Kb = torch.where(col[:, None, None], K[b], torch.zeros_like(K[b]))
        Vb = torch.where(col[:, None, None], V[b], torch.zeros_like(V[b]))
        s = (torch.einsum("ihd,jhd->hij", Qb, Kb) * sc).masked_fill(~ok, -math.inf)
        p = torch.softmax(s, -1).nan_to_num(0.0)
        dp = torch.einsum("ihd,jhd->hij", D_o, Vb)
        Ob = torch.where(row[:, None, None], O[b], torch.zeros_like(O[b]))
        D = torch.einsum("ihd,ihd->hi", D_o, Ob)
        D_abs = torch.einsum("ihd,ihd->hi", D_o.abs(), Ob.abs())
        ds = p * (dp - D[..., None])
        e_dp = 4 * dk * 2.0 ** -24 * torch.einsum("ihd,jhd->hij", D_o.abs(), Vb.abs())
        E = (2.02 * u + 2 * c) * ds.abs() + p * (e_dp + ((1.01 * u + c + 2.0 ** -20) * D_abs)[..., None])
        P_err = (u + c) * p
        if dt == torch.float16:
            P_err = P_err + 2.0 ** -33 * ok
            E = E + ok * (2.0 ** -29 * D_o.abs().max() + 2.0 ** -33 * (dp - D[..., None]).abs())
        bq[b] = torch.einsum("hij,jhd->ihd", E, Kb.abs()) * sc
        bk[b] = torch.einsum("hij,ihd->jhd", E, Qb.abs()) * sc
        bv[b] = torch.einsum("hij,ihd->jhd", P_err, D_o.abs())
    fold = (B, nkv, hkv, g, dk)
    return u, bq, bk.view(fold).sum(3), bv.view(fold).sum(3)


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
    (1, 1537, 1537, 2, 1, 64, 5000, 0, "bf16", [1400], False),
    (1, 2048, 2048, 1, 1, 128, 256, 4, "bf16", None, True),
    (1, 512, 512, 1, 1, 64, 255, 200, "bf16", None, False),
    (1, 3000, 3000, 4, 1, 64, 200, 4, "f16", [2999], False),      # sinks cut into parts
    (13, 900, 900, 9, 3, 128, 150, 3, "bf16", list(range(0, 910, 70)), False),
    (15, 1000, 1030, 7, 7, 128, 260, 200, "f16", None, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:9])))
def test_window_backward_against_the_formulas(case):
    B, nq, nkv, h, hkv, dk, window, sinks, dt, lens, packed = case
    q, k, v = inputs(1, B, nq, nkv, h, hkv, dk, DT[dt], packed)
    do = randn(gen(2), (B, nq, h, dk), DT[dt])
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, stats = forward(q, k, v, window, sinks, lt)
    ws = bpt.attn_window_backward_workspace(q, k, window, sinks)
    grads = tuple(torch.full(x.shape, math.nan, dtype=x.dtype, device="cuda") for x in (q, k, v))
    got = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, lens=lt, grads=grads, ws=ws)
    assert got is grads
    no_fault(ws)
    want = window_attention_grads(q.double(), k.double(), v.double(), do.double(), window, sinks,
                                  lens)
    u, *bound = grad_bounds(q, k, v, o, do, window, sinks, lens)
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        err = (g.double() - w).abs()
        tol = b + u * w.abs() * 1.01 + 2.0 ** -24
        assert (err <= tol).all(), (name, (err / tol).max().item(), (err - tol).max().item())
    again = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, lens=lt)
    for a, b in zip(got, again):
        assert torch.equal(a, b)  # the same bits every time


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_padding_may_hold_anything(dt):
    """Rows past the lengths hold NaN in every input: the gradients are those
    of clean padding, bitwise, and zeros in the padding."""
    dt = DT[dt]
    B, n, h, hkv, dk, window, sinks, lens = 3, 400, 4, 2, 64, 90, 3, [400, 130, 1]
    q, k, v = inputs(3, B, n, n, h, hkv, dk, dt)
    do = randn(gen(4), (B, n, h, dk), dt)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, stats = forward(q, k, v, window, sinks, lt)
    want = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, lens=lt)
    q2, k2, v2, o2, do2 = (x.clone() for x in (q, k, v, o, do))
    for b in range(B):
        for x in (q2, k2, v2, o2, do2):
            x[b, lens[b]:] = math.nan
    o3, stats3 = forward(q2, k2, v2, window, sinks, lt)
    assert torch.equal(o3, o) and torch.equal(stats3, stats)
    got = bpt.attn_window_backward(q2, k2, v2, o2, stats, do2, window, sinks, lens=lt)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
        for b in range(B):
            assert (g[b, lens[b]:] == 0).all()


def test_short_windows_with_sinks_and_padding():
    """A sequence shorter than a tile whose window has left its first keys."""
    q, k, v = inputs(5, 1, 60, 260, 2, 1, 64, torch.bfloat16)
    do = randn(gen(6), q.shape, q.dtype)
    lens = [215]
    for x in (k, v):
        x[0, 215:] = math.nan
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, stats = forward(q, k, v, 10, 6, lt)
    got = bpt.attn_window_backward(q, k, v, o, stats, do, 10, 6, lens=lt)
    kz, vz = k.clone(), v.clone()
    for x in (kz, vz):
        x[0, 215:] = 0
    want = window_attention_grads(q.double(), kz.double(), vz.double(), do.double(), 10, 6, lens)
    u, *bound = grad_bounds(q, kz, vz, o, do, 10, 6, lens)
    for g, w, b in zip(got, want, bound):
        assert ((g.double() - w).abs() <= b + 1.01 * u * w.abs() + 2.0 ** -24).all()


@pytest.mark.parametrize("scale", [1e-4, 300.0])
def test_fp16_gradients_of_any_scale(scale):
    """Small and large output gradients keep their relative accuracy."""
    q, k, v = inputs(7, 1, 700, 700, 2, 1, 128, torch.float16)
    do = randn(gen(8), q.shape, q.dtype, scale)
    o, stats = forward(q, k, v, 1000, 0, None)
    got = bpt.attn_window_backward(q, k, v, o, stats, do, 1000, 0)
    want = window_attention_grads(q.double(), k.double(), v.double(), do.double(), 1000, 0)
    u, *bound = grad_bounds(q, k, v, o, do, 1000, 0, None)
    for g, w, b in zip(got, want, bound):
        assert torch.isfinite(g).all()
        assert ((g.double() - w).abs() <= b + 1.01 * u * w.abs() + 2.0 ** -24).all()


def test_gradients_against_differences():
    """Directional differences of the fp64 forward against the kernels'
    gradients, within the sum of the elementwise bounds."""
    B, n, h, hkv, dk, window, sinks, lens = 1, 300, 4, 2, 64, 70, 3, [280]
    q, k, v = inputs(9, B, n, n, h, hkv, dk, torch.float16)
    do = randn(gen(10), q.shape, q.dtype)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, stats = forward(q, k, v, window, sinks, lt)
    got = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, lens=lt)
    u, *bound = grad_bounds(q, k, v, o, do, window, sinks, lens)
    x64 = [x.double() for x in (q, k, v)]
    loss = lambda xs: (window_attention(*xs, window, sinks, lens)[0] * do.double()).sum().item()
    g = gen(11)
    for i in range(3):
        d = torch.randn(x64[i].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-5
        up, down = list(x64), list(x64)
        up[i], down[i] = x64[i] + eps * d, x64[i] - eps * d
        diff = (loss(up) - loss(down)) / (2 * eps)
        dot = (got[i].double() * d).sum().item()
        tol = ((bound[i] + 1.01 * u * got[i].double().abs() + 2.0 ** -24) * d.abs()).sum().item()
        assert abs(diff - dot) <= tol + 1e-5 * abs(diff), (i, diff, dot, tol)


def test_packed_gradients_streams_and_graphs():
    """Gradients into the parts of one packed tensor, on another stream and
    from a captured graph: bitwise what the plain call gives."""
    B, n, h, dk, window, sinks = 2, 300, 3, 64, 100, 4
    q, k, v = inputs(12, B, n, n, h, h, dk, torch.bfloat16, packed=True)
    do = randn(gen(13), (B, n, h, dk), q.dtype)
    o, stats = forward(q, k, v, window, sinks, None)
    want = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks)
    dqkv = torch.full((B, n, 3, h, dk), math.nan, dtype=q.dtype, device="cuda")
    parts = (dqkv[:, :, 0], dqkv[:, :, 1], dqkv[:, :, 2])
    ws = bpt.attn_window_backward_workspace(q, k, window, sinks)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, grads=parts, ws=ws, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(parts, want):
        assert torch.equal(a, b)
    dqkv.fill_(math.nan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, grads=parts, ws=ws)
    for _ in range(2):
        graph.replay()
    for a, b in zip(parts, want):
        assert torch.equal(a, b)
    no_fault(ws)

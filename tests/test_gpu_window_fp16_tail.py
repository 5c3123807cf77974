"""Windowed attention in fp16 in which one key outweighs every other by far:
the many small weights keep their part of the output."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import window_attention
from test_gpu_window import gen, no_fault, randn

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.mark.parametrize("gap", [12.4, 22.6, 25.1, 29.3])  # bits between the peak and the rest
@pytest.mark.parametrize("dk,at,window,sinks", [(64, 0, 30000, 0), (128, 0, 19000, 1),
                                                (128, 5000, 30000, 0), (64, 19500, 30000, 0)])
def test_a_long_flat_tail_under_one_peak(gap, dk, at, window, sinks):
    nq, nkv, h = 130, 20000, 2
    k = torch.zeros((1, nkv, 1, dk), dtype=F16, device="cuda")
    k[0, at, 0, 0] = gap * math.log(2) * math.sqrt(dk) / 8
    v = randn(gen(51), (1, nkv, 1, dk), F16) + 100
    v[0, at] = 0
    q = randn(gen(52), (1, nq, h, dk), F16)
    q[..., 0] = 8
    stats = torch.empty((1, h, nq, 2), device="cuda")
    ws = bpt.attn_window_workspace(q, k, window, sinks)
    out = bpt.attn_window_forward(q, k, v, window, sinks, stats=stats, ws=ws)
    no_fault(ws)
    o, m, l, A = window_attention(q.double(), k.double(), v.double(), window, sinks)
    # (relative error of a weight as in ``bounds``; one column has all products,
    # whose magnitudes add up to the peak's score at most)
    u = torch.finfo(F16).eps / 2
    c = 2 * (2 * dk * 2.0 ** -24 * 1.01 * gap * math.log(2)) + 2 * 7.6e-5 + nkv * 2.0 ** -23
    # an fp16 weight is off by half a step, or (below 2^-25 of the reference) by
    # 2^-34 of it: P is held 2^9 times as large, the smallest step is 2^-24
    tol = (u + c) * A * (1 + u) + u * o.abs() + nkv * 2.0 ** -34 * v.abs().max() + 2.0 ** -25
    err = (out.double() - o).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    rel = (stats[..., 1].double() * torch.exp(stats[..., 0].double() - m) / l - 1).abs()
    assert (rel <= c + 2.0 ** -20).all(), rel.max().item()


@pytest.mark.parametrize("dk", [64, 128])
def test_large_scores_stay_finite(dk):
    """Scores of 10^7, whose last bit is a factor of two in a weight: the largest
    one wins, and no weight leaves the range of fp16."""
    n = 900
    u = torch.finfo(F16).eps / 2
    q = torch.full((1, n, 2, dk), 1000.0, dtype=F16, device="cuda")
    k = torch.randint(1, 1000, (1, n, 1, 1), generator=gen(53), device="cuda").to(F16)
    k = k.expand(1, n, 1, dk).contiguous()
    v = randn(gen(54), k.shape, F16)
    out = bpt.attn_window_forward(q, k, v, 300)
    for i in (0, 1, 130, 299, 300, 640, 899):
        lo = max(0, i - 299)
        row = k[0, lo:i + 1, 0, 0]
        if (row == row.max()).sum() == 1:
            best = v[0, lo + row.argmax()].double()
            # the weight is rounded once, the output once
            assert ((out[0, i].double() - best).abs() <= 2.02 * u * best.abs() + 2.0 ** -25).all(), i

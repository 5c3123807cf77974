"""Windowed attention over values that are not finite: what a row sees reaches
it, wherever the key falls in a tile and whatever its weight."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import window_attention
from test_gpu_window import DT, bounds, inputs, no_fault

pytestmark = pytest.mark.gpu
TYPES = [("bf16", 64), ("f16", 64), ("bf16", 128), ("f16", 128)]


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dt,dk", TYPES)
def test_a_bad_key_reaches_every_row_that_sees_it(dt, dk, bad):
    """One key of each head holds NaN, or gives the score +inf (whose softmax is
    NaN), the heads' keys at every column of a 128-key tile; the window is long
    enough for tiles that a whole block of rows sees."""
    B, h, n, window = 8, 16, 1024, 600
    q, k, v = inputs(21, B, n, n, h, h, dk, DT[dt])
    q[..., 0] = q[..., 0].abs() + 0.5
    clean = bpt.attn_window_forward(q, k, v, window)
    key = 300 + torch.arange(B * h, device="cuda").view(B, h)
    k2 = k.clone()
    for b in range(B):
        k2[b, key[b], torch.arange(h, device="cuda"), 0] = bad
    stats = torch.empty((B, h, n, 2), device="cuda")
    ws = bpt.attn_window_workspace(q, k2, window)
    out = bpt.attn_window_forward(q, k2, v, window, stats=stats, ws=ws)
    no_fault(ws)
    gap = torch.arange(n, device="cuda")[None, :, None] - key[:, None, :]
    hit = (gap >= 0) & (gap < window)
    assert out[hit].isnan().all(), hit[~out.isnan().all(-1) & hit].numel()
    assert stats[..., 1].transpose(1, 2)[hit].isnan().all()
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("dt,dk", TYPES)
def test_a_score_of_minus_infinity_is_a_weight_of_zero(dt, dk):
    n, window = 700, 600
    q, k, v = inputs(22, 1, n, n, 2, 2, dk, DT[dt])
    q[..., 0] = q[..., 0].abs() + 0.5
    u, c = bounds(q, k, DT[dt], window)
    k[0, 200::37, :, 0] = -math.inf
    out = bpt.attn_window_forward(q, k, v, window)
    o, _, _, A = window_attention(q.double(), k.double(), v.double(), window, 0)
    tiny = 2.0 ** -25 * window * v.abs().max().item() if dt == "f16" else 0
    tol = (u + c) * A * (1 + u) + u * o.abs() + 2.0 ** -25 + tiny
    assert ((out.double() - o).abs() <= tol).all()

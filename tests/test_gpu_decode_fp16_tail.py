"""One-token attention over an fp16 cache in which one slot outweighs every
other by far: the many small weights keep their part of the output."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import decode_attention
from test_gpu_cache import Pool, decode_bounds, gen, no_fault, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gap", [12.4, 22.6, 25.1, 29.3])  # bits between the peak and the rest
@pytest.mark.parametrize("dk,g,at", [(64, 1, 0), (128, 4, 0), (128, 12, 777), (64, 8, 1999)])
def test_a_long_flat_tail_under_one_peak(gap, dk, g, at):
    """More (sequence, kv head) pairs than blocks, so that the slots beside the
    peak share its reference."""
    B, hkv, n = 40, 16, 2000
    pool = Pool(1, [n] * B, hkv, dk, 64, torch.float16)
    pool.k.zero_()
    pool.v.copy_(randn(gen(2), pool.v.shape, torch.float16) + 100)
    page, row = pool.table[:, at // 64].long(), at % 64
    pool.k[page, :, row, 0] = gap * math.log(2) * math.sqrt(dk) / 8
    pool.v[page, :, row] = 0
    q = randn(gen(3), (B, hkv * g, dk), torch.float16)
    q[..., 0] = 8
    acc = torch.zeros((B, hkv, pool.cap), device="cuda")
    ws = bpt.attn_decode_workspace(q, pool.k, pool.table, True)
    out = bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens, acc=acc, ws=ws)
    no_fault(ws)
    assert torch.equal(out, bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens))
    for b in (0, 17, 39):
        k, v = pool.rows(pool.k, b, range(n)), pool.rows(pool.v, b, range(n))
        o, p, A = decode_attention(q[b].double(), k, v)
        u, c = decode_bounds(q[b].double(), k, n, torch.float16)
        # an fp16 weight is off by half a step, or (below 2^-25 of the reference) by
        # 2^-36 of it: P is held 2^11 times as large, the smallest step is 2^-24
        tol = (u + c) * A * (1 + u) + u * o.abs() + n * 2.0 ** -36 * v.abs().max() + 2.0 ** -25
        err = (out[b].double() - o).abs()
        assert (err <= tol).all(), (err / tol).max().item()
        w = p.view(hkv, g, n).sum(1)
        assert ((acc[b, :, :n].double() - w).abs() <= c * w + (g + 1) * 2.0 ** -24 * w).all()


def test_large_scores_stay_finite():
    """Scores of 10^7, whose last bit is a factor of two in a weight: the largest
    one wins, and no weight leaves the range of fp16."""
    pool = Pool(4, [700], 2, 128, 16, torch.float16)
    u = torch.finfo(torch.float16).eps / 2
    q = torch.full((1, 4, 128), 1000.0, dtype=torch.float16, device="cuda")
    pool.k.copy_(torch.randint(1, 1000, (*pool.k.shape[:3], 1), generator=gen(5), device="cuda")
                 .expand_as(pool.k))
    out = bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens)
    k, v = pool.rows(pool.k, 0, range(700)), pool.rows(pool.v, 0, range(700))
    for t in range(4):
        row = k[:, t // 2, 0]
        if (row == row.max()).sum() == 1:
            best = v[row.argmax(), t // 2]
            # the weight is rounded once, the output once
            assert ((out[0, t].double() - best).abs() <= 2.02 * u * best.abs() + 2.0 ** -25).all()

"""One-token attention over a slot whose score is NaN or +inf: the softmax is
NaN, in the output and in every accumulated weight."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from test_gpu_cache import DT, Pool, gen, no_fault, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dt,dk,h,lens,slot", [("bf16", 64, 4, [300, 90], 37),
                                               ("f16", 128, 24, [9000, 90], 8990),
                                               ("f16", 64, 2, [1, 90], 0)])
def test_a_bad_score_reaches_the_output_and_every_weight(bad, dt, dk, h, lens, slot):
    hkv, g = 2, h // 2
    pool = Pool(61, lens, hkv, dk, 16, DT[dt])
    q = randn(gen(62), (2, h, dk), DT[dt])
    q[..., 0] = q[..., 0].abs() + 0.5
    acc = torch.rand((2, hkv, pool.cap), generator=gen(63), device="cuda")
    run = lambda out: bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens, acc=acc,
                                      acc_out=out, ws=ws)
    ws = bpt.attn_decode_workspace(q, pool.k, pool.table, True)
    clean_acc = torch.zeros_like(acc)
    clean = run(clean_acc)
    pool.k[pool.table[0, slot // 16].long(), 1, slot % 16, 0] = bad
    got_acc = torch.zeros_like(acc)
    got = run(got_acc)
    no_fault(ws)
    assert got[0, g:].isnan().all() and got_acc[0, 1, :lens[0]].isnan().all()
    assert torch.equal(got[0, :g], clean[0, :g]) and torch.equal(got[1], clean[1])
    got_acc[0, 1, :lens[0]] = clean_acc[0, 1, :lens[0]]
    assert torch.equal(got_acc, clean_acc)

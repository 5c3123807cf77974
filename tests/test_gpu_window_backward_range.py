"""fp16 gradients of windowed attention over the range of V and dO: dS is held
in fp16 scaled by a power of two that follows both, per (sequence, kv head)."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import window_attention_grads, window_mask
from test_gpu_window import gen, inputs, no_fault, randn
from test_gpu_window_backward import forward, grad_bounds

pytestmark = pytest.mark.gpu
F16 = torch.float16


def pair_bounds(q, k, v, o, do, window, sinks, lens):
    """grad_bounds of each (sequence, kv head) by itself, and what dS loses in
    the subnormals: with R = max |dO_i| max |v_j| (2-norms; |dP - D| <= 2 R) dS
    is scaled by at least 2^13 / R, so a step of 2^-24 is off by 2^-38 R."""
    B, nq, h, dk = q.shape
    nkv, hkv = k.shape[1], k.shape[2]
    g = h // hkv
    sc = 1 / math.sqrt(dk)
    out = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v)]
    for b in range(B):
        n = nkv if lens is None else lens[b]
        ok = window_mask(nq, nkv, window, sinks, n, "cuda").double()
        rows = max(0, n - (nkv - nq))
        for t in range(hkv):
            hs, one = slice(t * g, (t + 1) * g), slice(b, b + 1)
            u, bq, bk, bv = grad_bounds(q[one, :, hs], k[one, :, t:t + 1], v[one, :, t:t + 1],
                                        o[one, :, hs], do[one, :, hs], window, sinks,
                                        None if lens is None else [n])
            if rows and n:
                R = (do[b, :rows, hs].double().norm(dim=-1).max()
                     * v[b, :n, t].double().norm(dim=-1).max()).item()
                lost = 2.0 ** -38 * R * sc
                bq += lost * (ok[:, :n] @ k[b, :n, t].double().abs())[None, :, None]
                bk += lost * (ok[:rows].T @ q[b, :rows, hs].double().abs().sum(1))[None, :, None]
            out[0][one, :, hs], out[1][one, :, t:t + 1], out[2][one, :, t:t + 1] = bq, bk, bv
    return u, out


def check(q, k, v, do, window, sinks, lens=None):
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, stats = forward(q, k, v, window, sinks, lt)
    ws = bpt.attn_window_backward_workspace(q, k, window, sinks)
    got = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, lens=lt, ws=ws)
    no_fault(ws)
    want = window_attention_grads(q.double(), k.double(), v.double(), do.double(), window, sinks,
                                  lens)
    u, bound = pair_bounds(q, k, v, o, do, window, sinks, lens)
    for name, x, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        assert torch.isfinite(x).all(), name
        err, tol = (x.double() - w).abs(), b + 1.01 * u * w.abs() + 2.0 ** -24
        assert (err <= tol).all(), (name, (err / tol).max().item())


@pytest.mark.parametrize("dk", [64, 128])
def test_large_values_of_one_sign_per_key(dk):
    """V is +400 or -400 in every column of a key and dO is 1: dP is +-400 d_k
    and dS up to half of it, which fp16 holds, but not 16 times as much."""
    q, k, _ = inputs(41, 2, 300, 300, 4, 2, dk, F16)
    sign = torch.tensor([1.0, -1.0], device="cuda").repeat(150)
    v = (400.0 * sign)[None, :, None, None].expand(2, 300, 2, dk).to(F16).contiguous()
    check(q, k, v, torch.ones_like(q), 1000, 0)


@pytest.mark.parametrize("vs,ds", [(300.0, 10.0), (1e-2, 1e-2), (200.0, 1e-3), (1e-3, 200.0),
                                   (0.0, 1.0), (1.0, 0.0)])
def test_scales_of_values_and_output_gradients(vs, ds):
    q, k, v = inputs(42, 2, 257, 400, 4, 2, 128, F16)
    do = randn(gen(43), q.shape, F16, ds)
    check(q, k, (v.float() * vs).to(F16), do, 150, 4, [400, 290])


def test_sequences_and_heads_of_different_scales():
    """A sequence, or a kv head, keeps its accuracy beside one whose output
    gradients are 2^19 times as large."""
    q, k, v = inputs(44, 3, 300, 300, 4, 2, 64, F16)
    do = torch.randn(q.shape, generator=gen(45), device="cuda")
    do[0] *= 2.0 ** -12
    do[1] *= 2.0 ** 7
    do[2, :, :2] *= 2.0 ** -12
    do[2, :, 2:] *= 2.0 ** 7
    check(q, k, v, do.to(F16), 90, 3)


def test_padding_does_not_set_the_scale():
    """Rows and keys past the lengths may hold anything: bitwise the gradients
    of clean padding."""
    lens = [300, 130, 1, 0]
    q, k, v = inputs(46, 4, 300, 300, 4, 2, 128, F16)
    do = randn(gen(47), q.shape, F16)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, stats = forward(q, k, v, 90, 3, lt)
    want = bpt.attn_window_backward(q, k, v, o, stats, do, 90, 3, lens=lt)
    for b, n in enumerate(lens):
        v[b, n:], do[b, n:] = 60000.0, math.inf
    got = bpt.attn_window_backward(q, k, v, o, stats, do, 90, 3, lens=lt)
    for a, w in zip(got, want):
        assert torch.equal(a, w)

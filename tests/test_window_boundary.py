"""Refusals of the windowed attention, reported before anything is enqueued
(no GPU needed; the addresses are never followed), and the fp64 definitions
against autograd and differences."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200 import build as bbuild
from oracle.attention import window_attention, window_attention_grads, window_mask

INV, UNS, WS = bpt.BPT_ERR_INVALID_ARG, bpt.BPT_ERR_UNSUPPORTED, bpt.BPT_ERR_WORKSPACE
BASE = 0x100000000


@pytest.fixture(scope="module", autouse=True)
def lib():
    bbuild.build()
    return bpt.load()


def addr(i):
    return BASE + i * 0x10000000


def win(**kw):
    f = dict(batch=2, n_q=300, n_kv=400, heads=4, kv_heads=2, d_k=64, window=100, sinks=4,
             dtype=bpt.BPT_BF16, reserved=0)
    f.update(kw)
    return bpt.Window(*f.values())


def rows(i, n, h, dk=64, at=0, **kw):
    f = dict(data=addr(i) + at, stride_b=n * h * dk, stride_n=h * dk, stride_h=dk)
    f.update(kw)
    return bpt.Rows(*f.values())


def args():
    return dict(w=win(), q=rows(0, 300, 4), k=rows(1, 400, 2), v=rows(2, 400, 2),
                o=rows(3, 300, 4), stats=addr(4), d_o=rows(5, 300, 4), lens=addr(6),
                dq=rows(7, 300, 4), dk=rows(8, 400, 2), dv=rows(9, 400, 2), ws=addr(10),
                nbytes=1 << 27)


def fwd(**kw):
    a = args()
    a.update(kw)
    return bpt.bpt_attn_window_forward(a["w"], a["q"], a["k"], a["v"], a["lens"], a["o"],
                                       a["stats"], a["ws"], a["nbytes"], None)


def bwd(**kw):
    a = args()
    a.update(kw)
    return bpt.bpt_attn_window_backward(a["w"], a["q"], a["k"], a["v"], a["o"], a["stats"],
                                        a["d_o"], a["lens"], a["dq"], a["dk"], a["dv"], a["ws"],
                                        a["nbytes"], None)


@pytest.mark.parametrize("fields,want", [
    (dict(dtype=bpt.BPT_F32), INV), (dict(dtype=5), INV), (dict(reserved=1), INV),
    (dict(batch=-1), INV), (dict(n_q=-1), INV), (dict(n_q=401), INV), (dict(heads=0), INV),
    (dict(kv_heads=3), INV), (dict(kv_heads=0), INV), (dict(window=0), INV),
    (dict(window=-5), INV), (dict(sinks=-1), INV), (dict(d_k=96), UNS), (dict(d_k=32), UNS),
    (dict(n_kv=1 << 31), UNS), (dict(heads=1 << 31, kv_heads=1), UNS),
    (dict(n_kv=1 << 28, heads=1 << 20), UNS),
], ids=str)
def test_bad_sizes(fields, want):
    w = win(**fields)
    assert fwd(w=w) == want and bwd(w=w) == want
    assert bpt.bpt_attn_window_workspace_size(w)[0] == want
    assert bpt.bpt_attn_window_backward_workspace_size(w)[0] == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INV), (dict(k=rows(1, 400, 2, data=None)), INV),
    (dict(v=rows(2, 400, 2, at=8)), INV), (dict(q=rows(0, 300, 4, stride_h=60)), INV),
    (dict(k=rows(1, 400, 2, stride_b=0)), INV), (dict(k=rows(1, 400, 2, stride_h=0)), INV),
    (dict(v=rows(2, 400, 2, stride_n=-128)), INV), (dict(lens=addr(6) + 2), INV),
    (dict(stats=addr(4) + 4), INV), (dict(ws=None), INV), (dict(ws=addr(10) + 16), INV),
    (dict(nbytes=128), WS), (dict(ws=addr(0)), INV),
], ids=str)
def test_bad_inputs(kw, want):
    assert fwd(**kw) == want and bwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(o=rows(0, 300, 4)), INV), (dict(o=rows(1, 300, 4, at=4096)), INV),
    (dict(o=rows(3, 300, 4, stride_n=64)), INV), (dict(o=None), INV),
    (dict(stats=addr(3)), INV), (dict(stats=addr(2)), INV),
], ids=str)
def test_bad_forward_outputs(kw, want):
    assert fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dq=rows(0, 300, 4)), INV), (dict(dk=rows(8, 400, 2, stride_n=64)), INV),
    (dict(dv=rows(8, 400, 2)), INV), (dict(dv=None), INV), (dict(stats=None), INV),
    (dict(d_o=rows(5, 300, 4, stride_b=0)), INV), (dict(dq=rows(10, 300, 4)), INV),
    (dict(nbytes=4096), WS), (dict(w=win(n_q=0)), INV), (dict(w=win(batch=70000)), UNS),
    (dict(w=win(batch=40000)), UNS),
], ids=str)
def test_bad_backwards(kw, want):
    assert bwd(**kw) == want


def test_empty_work_is_done():
    assert fwd(w=win(batch=0)) == bwd(w=win(batch=0)) == bpt.BPT_OK
    assert fwd(w=win(n_q=0)) == bpt.BPT_OK
    assert bwd(w=win(n_q=0, n_kv=0)) == bpt.BPT_OK


def test_backward_workspace_holds_terms_and_parts():
    # one kv head, many queries that see the sinks: the first block is cut
    _, small = bpt.bpt_attn_window_backward_workspace_size(win(sinks=0))
    assert small <= 4096 + 2 * 4 * 300 * 8 + 512
    w = win(batch=1, n_q=65536, n_kv=65536, heads=1, kv_heads=1, window=256, sinks=4)
    _, big = bpt.bpt_attn_window_backward_workspace_size(w)
    assert 65536 * 8 + 2 * 2 * 128 * 64 * 4 < big < 65536 * 8 + (80 << 20)


def test_front_end_refuses_tensors_that_do_not_fit():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bpt.attn_window_forward(q, q, q, 4)       # not on a GPU
    with pytest.raises(TypeError):
        bpt.attn_window_workspace(q.float(), q.float(), 4)
    with pytest.raises(ValueError):
        bpt.attn_window_workspace(q[0], q, 4)
    with pytest.raises(bpt.BptError):
        bpt.attn_window_workspace(q, q, 0)


@pytest.mark.parametrize("nq,nkv,h,hkv,window,sinks,lens", [
    (5, 5, 1, 1, 2, 0, None), (4, 9, 4, 2, 3, 2, [9, 6]), (7, 7, 2, 1, 20, 1, [0, 7]),
    (1, 6, 3, 3, 1, 3, None),
])
def test_the_definition_and_its_gradients(nq, nkv, h, hkv, window, sinks, lens):
    """The oracle's forward row by row from the words of its definition, its
    gradients against autograd and against differences."""
    torch.manual_seed(0)
    B, dk = (2 if lens else 1), 8
    q, do = (torch.randn(B, nq, h, dk, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(B, nkv, hkv, dk, dtype=torch.float64) for _ in range(2))
    o, m, l, A = window_attention(q, k, v, window, sinks, lens)
    for b in range(B):
        n = nkv if lens is None else lens[b]
        for i in range(nq):
            p = nkv - nq + i
            see = [j for j in range(nkv) if j <= p and p < n and (p - j < window or j < sinks)]
            assert window_mask(nq, nkv, window, sinks, n, "cpu")[i].nonzero().view(-1).tolist() == see
            for t in range(h):
                if not see:
                    assert (o[b, i, t] == 0).all() and m[b, t, i] == -math.inf and l[b, t, i] == 0
                    continue
                s = torch.stack([q[b, i, t] @ k[b, j, t // (h // hkv)] for j in see]) / math.sqrt(dk)
                w = torch.softmax(s, 0)
                want = sum(w[x] * v[b, j, t // (h // hkv)] for x, j in enumerate(see))
                assert torch.allclose(o[b, i, t], want, atol=1e-12)
                assert torch.allclose(m[b, t, i] + l[b, t, i].log(), torch.logsumexp(s, 0))
    got = window_attention_grads(q, k, v, do, window, sinks, lens)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    ok = torch.stack([window_mask(nq, nkv, window, sinks, nkv if lens is None else lens[b], "cpu")
                      for b in range(B)])
    s = torch.einsum("bihd,bjhd->bhij", leaves[0], leaves[1].repeat_interleave(h // hkv, 2))
    s = (s / math.sqrt(dk)).masked_fill(~ok[:, None], -1e300)
    w = torch.softmax(s, -1) * ok[:, None]
    out = torch.einsum("bhij,bjhd->bihd", w, leaves[2].repeat_interleave(h // hkv, 2))
    for g, a in zip(got, torch.autograd.grad(out, leaves, do)):
        assert torch.allclose(g, a, atol=1e-12)
    xs = [q, k, v]
    for i in range(3):
        d = torch.randn_like(xs[i])
        up, down = list(xs), list(xs)
        up[i], down[i] = xs[i] + 1e-6 * d, xs[i] - 1e-6 * d
        f = [(window_attention(*x, window, sinks, lens)[0] * do).sum() for x in (up, down)]
        assert abs((f[0] - f[1]) / 2e-6 - (got[i] * d).sum()) < 1e-7

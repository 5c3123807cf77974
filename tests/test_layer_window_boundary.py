"""Refusals of the windowed layer and of the decode step, before anything is
enqueued (no GPU needed; the addresses are never followed)."""
import pytest

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200 import build as bbuild

INV, UNS, WS = bpt.BPT_ERR_INVALID_ARG, bpt.BPT_ERR_UNSUPPORTED, bpt.BPT_ERR_WORKSPACE
BASE = 0x1000000000


@pytest.fixture(scope="module", autouse=True)
def lib():
    bbuild.build()
    return bpt.load()


def addr(i):
    return BASE + i * 0x10000000


PARAMS = [addr(i) for i in range(11)]


def cache(**kw):
    f = dict(k=addr(30), v=addr(31), page_table=addr(32), lens=addr(33), batch=2, pages=64,
             kv_heads=4, page_size=16, d_k=64, max_pages=20, dtype=bpt.BPT_F16, reserved=0)
    f.update(kw)
    return bpt.Cache(*f.values())


def fwd(B=2, N=300, d=256, h=4, d_ff=512, dtype=bpt.BPT_BF16, window=50, sinks=2, lens=addr(11),
        out=addr(12), stats=addr(13), o=addr(14), c=None, new_lens=None, acc=None, pos=None,
        seen=None, ws=addr(15), nbytes=1 << 27, params=PARAMS):
    return bpt.bpt_layer_forward_window(*params, B, N, d, h, d_ff, dtype, window, sinks, lens, out,
                                        stats, o, c, new_lens, acc, pos, seen, ws, nbytes, None)


def bwd(B=2, N=300, d=256, h=4, d_ff=512, dtype=bpt.BPT_BF16, window=50, sinks=2, lens=addr(11),
        stats=addr(13), o=addr(14), dZ=addr(16), ws=addr(15), nbytes=1 << 27, grads=None):
    grads = grads or [addr(17 + i) for i in range(11)]
    return bpt.bpt_layer_backward_window(*PARAMS, stats, o, dZ, B, N, d, h, d_ff, dtype, window,
                                         sinks, lens, *grads, ws, nbytes, None)


def dec(c=None, d=256, d_ff=512, window=0, sinks=0, acc=None, pos=None, seen=None,
        new_lens=addr(12), out=addr(13), ws=addr(15), nbytes=1 << 27, x=addr(0)):
    return bpt.bpt_layer_decode(x, addr(1), addr(2), addr(3), addr(4),
                                cache() if c is None else c, d, d_ff, window, sinks, acc, pos,
                                seen, new_lens, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), INV), (dict(window=-1), INV), (dict(sinks=-1), INV),
    (dict(dtype=bpt.BPT_F32), UNS), (dict(dtype=bpt.BPT_F16), INV), (dict(h=3), INV),
    (dict(d=96, h=3), UNS), (dict(lens=addr(11) + 2), INV), (dict(ws=addr(15) + 16), INV),
    (dict(nbytes=4096), WS), (dict(out=None), INV), (dict(out=addr(15)), INV),
    (dict(stats=addr(12)), INV), (dict(o=addr(12)), INV), (dict(lens=addr(12)), INV),
    (dict(new_lens=addr(20)), INV), (dict(c=cache()), INV),
    (dict(c=cache(batch=3), new_lens=addr(20)), INV),
    (dict(c=cache(kv_heads=2, d_k=128), new_lens=addr(20)), INV),
    (dict(c=cache(dtype=bpt.BPT_BF16), new_lens=addr(20)), INV),
    (dict(c=cache(), new_lens=addr(33)), INV), (dict(c=cache(k=addr(12)), new_lens=addr(20)), INV),
    (dict(c=cache(v=addr(15) + 4096), new_lens=addr(20)), INV),
    (dict(c=cache(), new_lens=addr(20), acc=addr(0)), INV),
    (dict(params=[addr(0) + 4] + PARAMS[1:]), INV),
], ids=str)
def test_bad_windowed_forwards(kw, want):
    assert fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(window=0), INV), (dict(sinks=-2), INV), (dict(dtype=bpt.BPT_F32), UNS),
    (dict(o=None), INV), (dict(stats=None), INV), (dict(dZ=None), INV), (dict(nbytes=1 << 16), WS),
    (dict(ws=addr(15) + 16), INV), (dict(lens=addr(15)), INV),
    (dict(grads=[addr(0)] + [addr(18 + i) for i in range(10)]), INV),
], ids=str)
def test_bad_windowed_backwards(kw, want):
    assert bwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(c=cache(dtype=bpt.BPT_BF16)), INV), (dict(d=512), INV), (dict(d_ff=500), UNS),
    (dict(c=cache(kv_heads=8, d_k=32)), UNS), (dict(window=-1), INV), (dict(sinks=-1), INV),
    (dict(new_lens=None), INV), (dict(new_lens=addr(33)), INV), (dict(out=None), INV),
    (dict(out=addr(15)), INV), (dict(ws=addr(15) + 64), INV), (dict(nbytes=4096), WS),
    (dict(acc=addr(13)), INV), (dict(pos=addr(30)), INV), (dict(x=addr(0) + 2), INV),
    (dict(c=cache(k=addr(15))), INV), (dict(c=cache(lens=addr(13))), INV),
    (dict(c=cache(batch=40000)), UNS), (dict(acc=addr(0)), INV), (dict(c=cache(k=addr(3))), INV),
], ids=str)
def test_bad_decode_steps(kw, want):
    assert dec(**kw) == want


def test_empty_calls_and_sizes():
    assert fwd(B=0) == bwd(B=0) == dec(c=cache(batch=0)) == bpt.BPT_OK
    st, n = bpt.bpt_layer_forward_window_workspace_size(2, 300, 256, 4, 512, bpt.BPT_BF16)
    _, plain = bpt.bpt_layer_workspace_size(2, 300, 256, 4, 512, 1, bpt.BPT_BF16)
    assert st == bpt.BPT_OK and n == plain + 2 * 300 * 256 * 2
    st, n = bpt.bpt_layer_decode_workspace_size(cache(), 256, 512, 0)
    _, with_acc = bpt.bpt_layer_decode_workspace_size(cache(), 256, 512, 1)
    assert st == bpt.BPT_OK and with_acc > n > (4 * 256 * 256 + 2 * 256 * 512) * 2
    ptrs = [addr(i) for i in range(6)]
    assert bpt.bpt_layer_decode_prepare(*ptrs, cache(), 256, 512, 0, addr(15), n - 1, None) == WS
    assert bpt.bpt_layer_decode_prepare(None, *ptrs[1:], cache(), 256, 512, 0, addr(15), n,
                                        None) == INV
    assert bpt.bpt_layer_decode_prepare(*ptrs, cache(), 256, 512, 0, addr(0), n, None) == INV

"""Refusals of the cache's operators: reported before anything is enqueued, so
they need no GPU (the addresses below are never followed)."""
import ctypes

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200 import build as bbuild
from oracle.attention import evict_order, visible_slots

INV, UNS, WS = bpt.BPT_ERR_INVALID_ARG, bpt.BPT_ERR_UNSUPPORTED, bpt.BPT_ERR_WORKSPACE
BASE = 0x100000000


@pytest.fixture(scope="module", autouse=True)
def lib():
    bbuild.build()
    return bpt.load()


def addr(i):
    return BASE + i * 0x10000000


def cache(**kw):
    f = dict(k=addr(0), v=addr(1), page_table=addr(2), lens=addr(3), batch=4, pages=64,
             kv_heads=2, page_size=16, d_k=64, max_pages=8, dtype=bpt.BPT_F16, reserved=0)
    f.update(kw)
    return bpt.Cache(*f.values())


BAD_CACHES = [
    (dict(dtype=bpt.BPT_F32), INV), (dict(dtype=9), INV), (dict(reserved=1), INV),
    (dict(batch=-1), INV), (dict(pages=0), INV), (dict(kv_heads=0), INV),
    (dict(page_size=0), INV), (dict(max_pages=0), INV), (dict(d_k=96), UNS),
    (dict(d_k=256), UNS), (dict(batch=70000), UNS), (dict(max_pages=1 << 28), UNS),
    (dict(pages=1 << 27), UNS), (dict(pages=1 << 40), UNS),
]
BAD_POINTERS = [(dict(k=None), INV), (dict(v=addr(1) + 8), INV), (dict(page_table=None), INV),
                (dict(lens=addr(3) + 2), INV), (dict(v=addr(0) + 16), INV)]


def append(c, k=addr(4), v=addr(5), tokens=3, strides=(384, 128, 64, 384, 128, 64), counts=None,
           new_lens=addr(6), acc=None, pos=None, seen=None, ws=addr(7), nbytes=1 << 20):
    s = (ctypes.c_int64 * 6)(*strides) if strides is not None else None
    return bpt.bpt_cache_append(c, k, v, tokens, s, counts, new_lens, acc, pos, seen, ws, nbytes,
                                None)


def decode(c, q=addr(4), heads=4, qs=(256, 64), window=0, sinks=0, acc=None, acc_out=None,
           out=addr(5), os=(256, 64), ws=addr(7), nbytes=1 << 27):
    return bpt.bpt_attn_decode(c, q, heads, *qs, window, sinks, acc, acc_out, out, *os, ws, nbytes,
                               None)


def evict(c, budget=5, recent=1, sinks=1, acc=addr(4), pos=addr(5), seen=addr(6), acc_out=addr(4),
          pos_out=addr(5), new_lens=addr(3), ws=addr(7), nbytes=1 << 27):
    return bpt.bpt_cache_evict(c, budget, recent, sinks, acc, pos, seen, acc_out, pos_out,
                               new_lens, ws, nbytes, None)


@pytest.mark.parametrize("fields,want", BAD_CACHES + BAD_POINTERS, ids=str)
def test_bad_caches(fields, want):
    c = cache(**fields)
    assert append(c) == want and decode(c) == want and evict(c) == want
    if (fields, want) in BAD_CACHES:
        assert bpt.bpt_cache_workspace_size(c)[0] == want
        assert bpt.bpt_attn_decode_workspace_size(c, 4, 0)[0] == want


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INV), (dict(k=None), INV), (dict(v=addr(5) + 4), INV),
    (dict(strides=None), INV), (dict(strides=(384, 128, 60, 384, 128, 64)), INV),
    (dict(strides=(384, 128, 64, -8, 128, 64)), INV), (dict(new_lens=None), INV),
    (dict(new_lens=addr(3)), INV), (dict(acc=addr(0)), INV), (dict(pos=addr(4) + 1), INV),
    (dict(k=addr(0) + 4096), INV), (dict(ws=None), INV), (dict(ws=addr(7) + 16), INV),
    (dict(nbytes=4095), WS), (dict(tokens=1 << 30), UNS), (dict(counts=addr(6)), INV),
    (dict(seen=addr(6)), INV), (dict(acc=addr(8), pos=addr(8)), INV),
], ids=str)
def test_bad_appends(kw, want):
    assert append(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(heads=0), INV), (dict(heads=3), INV), (dict(heads=1024), UNS), (dict(q=None), INV),
    (dict(q=addr(4) + 8), INV), (dict(out=None), INV), (dict(qs=(256, 60)), INV),
    (dict(os=(256, 32)), INV), (dict(os=(64, 64)), INV), (dict(window=-1), INV),
    (dict(sinks=-1), INV), (dict(acc=addr(8)), INV), (dict(acc_out=addr(8)), INV),
    (dict(acc=addr(8), acc_out=addr(8) + 64), INV), (dict(acc=addr(8), acc_out=addr(4)), INV),
    (dict(out=addr(4)), INV), (dict(out=addr(1) + 1024), INV), (dict(nbytes=1000), WS),
    (dict(ws=addr(7) + 128), INV), (dict(ws=addr(0)), INV),
], ids=str)
def test_bad_decodes(kw, want):
    assert decode(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(budget=0), INV), (dict(recent=-1), INV), (dict(sinks=-1), INV), (dict(acc=None), INV),
    (dict(pos=None), INV), (dict(seen=None), INV), (dict(new_lens=None), INV),
    (dict(acc_out=addr(4) + 4), INV), (dict(pos_out=addr(4)), INV), (dict(new_lens=addr(6)), INV),
    (dict(new_lens=addr(3) + 4), INV), (dict(nbytes=4096), WS), (dict(ws=addr(4)), INV),
    (dict(acc=addr(0), acc_out=addr(0)), INV),
], ids=str)
def test_bad_evictions(kw, want):
    assert evict(cache(), **kw) == want


def test_empty_batches_do_nothing():
    c = cache(batch=0)
    assert append(c) == decode(c) == evict(c) == bpt.BPT_OK


def test_workspace_sizes():
    st, a = bpt.bpt_cache_workspace_size(cache())
    assert st == bpt.BPT_OK and a >= 4096 + 4 * 4 * 2 * 128
    st, b = bpt.bpt_attn_decode_workspace_size(cache(), 8, 0)
    st2, c = bpt.bpt_attn_decode_workspace_size(cache(), 8, 1)
    assert st == st2 == bpt.BPT_OK and c - b >= 4 * 8 * 128 * 4
    assert decode(cache(), nbytes=b - 1) == WS


def test_front_end_refuses_tensors_that_do_not_fit():
    kc = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        bpt.attn_decode(q, kc, kc, table, lens)            # not on a GPU
    with pytest.raises(TypeError):
        bpt.cache_workspace(kc.float(), table)
    with pytest.raises(ValueError):
        bpt.cache_workspace(kc[0], table)


def test_the_definitions_small_cases():
    assert visible_slots(5, 0, 0) == [0, 1, 2, 3, 4]
    assert visible_slots(6, 2, 1) == [0, 4, 5] and visible_slots(0, 2, 1) == []
    # budget 3 of 5: slot 4 (recent) and the two largest, ties to the lowest
    assert evict_order([1.0, 3.0, 1.0, 0.0, 0.0], [0, 1, 2, 3, 4], 5, 3, 1, 0) == [0, 1, 4]
    assert evict_order([0.0, 3.0, 1.0, 0.0, 5.0], [0, 1, 2, 3, 4], 5, 2, 0, 0) == [4, 1]
    assert evict_order([1.0], [0], 1, 4, 0, 0) == [0]

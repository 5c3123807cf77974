"""Gradients of the windowed attention that share elements with one another are
refused before anything is enqueued; interleaved ones are not (no GPU needed:
a call that passes is stopped by its workspace, which is too small)."""
import itertools
import random

import pytest

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200 import build as bbuild

INV, WS = bpt.BPT_ERR_INVALID_ARG, bpt.BPT_ERR_WORKSPACE
BASE = 0x100000000


@pytest.fixture(scope="module", autouse=True)
def lib():
    bbuild.build()
    return bpt.load()


def rows(at, strides, base=BASE):
    return bpt.Rows(base + 2 * at, *strides)


def call(dq, dk, dv, B=2, nq=6, nkv=9, h=4, hkv=2, dk_=64):
    """The backward's status with these gradients and a workspace of a header."""
    w = bpt.Window(B, nq, nkv, h, hkv, dk_, 5, 1, bpt.BPT_BF16, 0)
    far = lambda i, n, heads: rows(0, (n * heads * dk_, heads * dk_, dk_), BASE + (i << 32))
    st, need = bpt.bpt_attn_window_backward_workspace_size(w)
    assert st == bpt.BPT_OK and need > 4096
    return bpt.bpt_attn_window_backward(w, far(1, nq, h), far(2, nkv, hkv), far(3, nkv, hkv),
                                        far(4, nq, h), BASE + (5 << 32), far(6, nq, h), None, dq, dk,
                                        dv, BASE + (7 << 32), 4096, None)


def elements(r, counts, dk):
    at = (r.data - BASE) // 2
    s = (r.stride_b, r.stride_n, r.stride_h)
    out = set()
    for i in itertools.product(*map(range, counts)):
        a = at + sum(x * y for x, y in zip(i, s))
        out.update(range(a, a + dk, 8))
    return out


def test_packed_gradients_pass():
    n, h, d = 9, 4, 64
    s = (n * 3 * h * d, 3 * h * d, d)                   # [B, N, 3, h, dk]
    parts = [rows(i * h * d, s) for i in range(3)]
    assert call(*parts, nq=n, hkv=h) == WS
    s = (n * 3 * h * d, 3 * h * d, 3 * d)               # [B, N, h, 3, dk]
    assert call(*[rows(i * d, s) for i in range(3)], nq=n, hkv=h) == WS
    s = (n * 8 * d, 8 * d, d)                           # [B, N, h + 2 hkv, dk]
    assert call(rows(0, s), rows(4 * d, s), rows(6 * d, s), nq=n) == WS
    s = (3 * h * n * d, d, n * d)                       # [B, 3, h, N, dk]
    assert call(*[rows(i * h * n * d, s) for i in range(3)], nq=n, hkv=h) == WS
    # one buffer per sequence, dq before dk before dv, each of its own strides
    b = (6 * 4 + 2 * 9 * 2) * d
    assert call(rows(0, (b, 4 * d, d)), rows(24 * d, (b, 2 * d, d)),
                rows(42 * d, (b, 2 * d, d))) == WS


@pytest.mark.parametrize("shift", [0, 8, 64, 256, 24 * 64 - 8])
def test_gradients_that_share_rows_are_refused(shift):
    sq, sk = (6 * 4 * 64, 4 * 64, 64), (9 * 2 * 64, 2 * 64, 64)
    apart = rows(1 << 20, sk)
    assert call(rows(0, sq), rows(shift, sk), apart) == INV
    assert call(rows(0, sq), apart, rows(shift, sk)) == INV
    assert call(rows(1 << 20, sq), rows(0, sk), rows(shift, sk)) == INV
    assert call(rows(1 << 20, sq), rows(shift, sk), rows(0, sk)) == INV


def test_random_layouts_against_their_elements():
    """Layouts in any order of the dimensions, with and without room between
    them, at offsets that interleave or collide: refused exactly if two of the
    three tensors share an element."""
    rng = random.Random(5)
    seen = {INV: 0, WS: 0}
    for _ in range(600):
        B, nkv, hkv, g, d = (rng.randint(1, 3), rng.randint(1, 6), rng.randint(1, 3),
                             rng.randint(1, 2), rng.choice([64, 128]))
        nq, h = rng.randint(1, nkv), hkv * g
        room = rng.choice([1, 1, 3])

        def layout(counts, order, pad):
            s, ext = [0, 0, 0], d * pad
            for k in order:
                s[k] = ext
                ext = ext * counts[k] + rng.choice([0, 0, 8, d])
            return tuple(s), ext

        order = rng.sample(range(3), 3)
        cq, ck = (B, nq, h), (B, nkv, hkv)
        sq, eq = layout((B, nkv, h), order, room)
        if rng.random() < 0.6:
            sk, ek = sq, eq
        else:
            sk, ek = layout(ck, rng.choice([order, rng.sample(range(3), 3)]), room)
        offs = [rng.choice([0, d, 2 * d, h * d, sq[order[1]], sq[order[2]], eq, eq + ek,
                            8 * rng.randint(0, eq // 4)]) for _ in range(3)]
        r = [rows(offs[0], sq), rows(offs[1], sk), rows(offs[2], sk)]
        sets = [elements(r[0], cq, d), elements(r[1], ck, d), elements(r[2], ck, d)]
        meet = any(sets[i] & sets[j] for i, j in ((0, 1), (0, 2), (1, 2)))
        got = call(*r, B=B, nq=nq, nkv=nkv, h=h, hkv=hkv, dk_=d)
        assert got == (INV if meet else WS), (B, nq, nkv, h, hkv, d, sq, sk, offs)
        seen[got] += 1
    assert min(seen.values()) > 50, seen

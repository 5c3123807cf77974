"""Values of V that are not finite, in rows that see them and in rows that do
not: only the columns that hold them change, and the call stays short."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import window_attention, window_mask
from test_gpu_window import DT, bounds, inputs, no_fault

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,dk", [("bf16", 64), ("f16", 128), ("f16", 64), ("bf16", 128)])
def test_columns_of_bad_values(dt, dk):
    """NaN, an infinity of either sign and both signs, each in a column of its
    own: rows that see one get it there (whatever its weight: key 200's is
    e^-300 or less), all else stays within the roundings."""
    n, h, window, sinks = 900, 2, 300, 4
    dt = DT[dt]
    q, k, v = inputs(31, 1, n, n, h, 1, dk, dt)
    q[..., 0], k[..., 0] = 30.0, 0.0
    k[0, 200, 0, 0] = -math.sqrt(dk) * 10.0 - 30.0  # q.k / sqrt(dk) below -300 + 6 |k|
    u, c = bounds(q[..., 1:], k[..., 1:], dt, window + sinks)
    o, _, _, A = window_attention(q.double(), k.double(), v.double(), window, sinks)
    bad = [(2, 3, math.nan), (2, 7, -math.inf), (200, 11, math.nan), (200, 12, math.inf),
           (250, 13, math.inf), (260, 13, -math.inf), (250, 63, math.inf),
           (50, 20, math.nan), (60, 21, math.inf)]
    v2 = v.clone()
    for j, col, x in bad:
        v2[0, j, 0, col] = x
    ws = bpt.attn_window_workspace(q, k, window, sinks)
    out = bpt.attn_window_forward(q, k, v2, window, sinks, ws=ws)
    no_fault(ws)
    mask = window_mask(n, n, window, sinks, n, "cuda")
    want = o.clone()
    for j, col, x in bad:
        want[0, mask[:, j], :, col] += x  # inf - inf and NaN as the sum has them
    settled = ~torch.isfinite(want)
    assert (out.double()[settled].isnan() == want[settled].isnan()).all()
    inf = settled & ~want.isnan()
    assert (out.double()[inf] == want[inf]).all()
    tiny = 2.0 ** -25 * (window + sinks) * v.abs().max().item() if dt == torch.float16 else 0
    tol = (u + c) * A * (1 + u) + u * o.abs() + 2.0 ** -25 + tiny
    err = (out.double() - o).abs()
    assert (err <= tol)[~settled].all(), (err - tol)[~settled].max().item()


def test_whole_rows_of_bad_values():
    """Garbage behind the sinks, in the tile that they lie in, is seen by the
    first rows only."""
    n, h, window, sinks = 1500, 2, 200, 4
    q, k, v = inputs(32, 2, n, n, h, h, 64, torch.bfloat16)
    v2 = v.clone()
    v2[0, 50], v2[1, 90, 1] = math.nan, math.inf
    u, c = bounds(q, k, q.dtype, window + sinks)
    o, _, _, A = window_attention(q.double(), k.double(), v.double(), window, sinks)
    out = bpt.attn_window_forward(q, k, v2, window, sinks)
    mask = window_mask(n, n, window, sinks, n, "cuda")
    hit = torch.zeros(2, n, h, dtype=torch.bool, device="cuda")
    hit[0] |= mask[:, 50][:, None]
    hit[1, :, 1] |= mask[:, 90]
    assert out[0][hit[0]].isnan().all() and (out[1][hit[1]] == math.inf).all()
    tol = (u + c) * A * (1 + u) + u * o.abs() + 2.0 ** -25
    assert ((out.double() - o).abs() <= tol)[~hit].all()


@pytest.mark.parametrize("key,value", [(1, math.nan), (50, math.inf)], ids=["seen", "masked"])
def test_one_bad_value_leaves_the_call_short(key, value):
    """A NaN in a sink that every row sees, an infinity that shares its tile:
    all 16384 rows of a head are done again.  Key by key that is 4100 dependent
    steps for each of a warp's 32 rows, 71 ms in all; with the keys in parallel
    about a tenth."""
    n, h, window = 16384, 8, 4096
    q, k, v = inputs(33, 1, n, n, h, h, 64, torch.bfloat16)
    out, ws = torch.empty_like(q), bpt.attn_window_workspace(q, k, window, 4)

    def ms(values):
        times = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            bpt.attn_window_forward(q, k, values, window, 4, out=out, ws=ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean = ms(v)
    v[0, key, 0, 5] = value
    assert ms(v) <= clean + 12.0

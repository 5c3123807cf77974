"""Calls on a stream other than the current one, with nothing allocated by the
caller, and refusals of the layer forms that need tensors on a GPU."""
import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200.inputs import LayerShape, make_inputs

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def leave_rubbish():
    """Freed blocks of the current stream that hold set bits, and work still
    queued there that would hand them over late."""
    for n in (1 << 12, 1 << 16, 1 << 20, 1 << 24):
        torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20_000_000)


def on_side(call, fresh=lambda: ()):
    """call(None, ...) and call(a side stream, ...) while the current stream is
    busy, each on its own fresh() tensors."""
    one, two = fresh(), fresh()
    want = call(None, *one)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    leave_rubbish()
    got = call(side, *two)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip([*want, *one], [*got, *two]):
        assert torch.equal(a, b)


def tensors(seed, *shapes, dt=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(dt) for s in shapes]


def test_windowed_attention_on_another_stream():
    q, do, k, v = tensors(1, (2, 300, 4, 64), (2, 300, 4, 64), (2, 300, 2, 64), (2, 300, 2, 64))
    stats = torch.empty((2, 4, 300, 2), device="cuda")
    o = bpt.attn_window_forward(q, k, v, 90, 140, stats=stats)
    on_side(lambda s: [bpt.attn_window_forward(q, k, v, 90, 140, stream=s)])
    on_side(lambda s: bpt.attn_window_backward(q, k, v, o, stats, do, 90, 140, stream=s))


def test_cache_operators_on_another_stream():
    B, hkv, ps, per = 3, 2, 16, 90
    kc, vc = tensors(2, (B * per, hkv, ps, 128), (B * per, hkv, ps, 128))
    q, kn, vn = tensors(3, (B, 8, 128), (B, 5, hkv, 128), (B, 5, hkv, 128))
    table = torch.randperm(B * per, device="cuda").int().view(B, per)
    lens = torch.tensor([1400, 3, 700], dtype=torch.int32, device="cuda")
    acc = torch.rand((B, hkv, per * ps), device="cuda")
    pos = torch.arange(per * ps, dtype=torch.int32, device="cuda").expand_as(acc).contiguous()

    on_side(lambda s, k, v: [bpt.cache_append(kn, vn, k, v, table, lens, stream=s)],
            lambda: [kc.clone(), vc.clone()])
    on_side(lambda s, to: [bpt.attn_decode(q, kc, vc, table, lens, 500, 4, acc=acc, acc_out=to,
                                           stream=s)], lambda: [torch.zeros_like(acc)])
    on_side(lambda s, k, v, a, p, n: [bpt.cache_evict(k, v, table, n, a, p, lens, 200, 20, 4,
                                                      stream=s)],
            lambda: [kc.clone(), vc.clone(), acc.clone(), pos.clone(), lens.clone()])


def layer():
    cfg = LayerShape("side", B=2, N=200, d=256, h=4, d_ff=512, causal=True, dtype="bf16",
                     block=128, seed=71, ln_scale=0.1, bias_scale=0.2)
    dev = bpt.to_device(make_inputs(cfg), "bf16")
    return dev.pop("x"), dev


def test_layer_on_another_stream():
    x, p = layer()
    stats, o = torch.empty((2, 4, 200, 2), device="cuda"), tensors(5, x.shape, dt=torch.float16)[0]
    bpt.layer_forward_window(x, p, 4, 64, 4, stats=stats, keep_o=o)
    dz = tensors(6, x.shape, dt=torch.float32)[0]
    on_side(lambda s: bpt.layer_forward_window(x, p, 4, 64, 4, stream=s)[:1])
    on_side(lambda s: list(bpt.layer_backward_window(x, p, 4, 64, 4, stats, o, dz,
                                                     stream=s)[0].values()))
    kc, vc = tensors(7, (8, 4, 32, 64), (8, 4, 32, 64), dt=torch.float16)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([100, 5], dtype=torch.int32, device="cuda")
    token = x[:, 0].contiguous()

    def step(s, k, v):
        ws = bpt.layer_decode_workspace(p, k, table, stream=s)
        return bpt.layer_decode(token, p, k, v, table, lens, ws, stream=s)

    on_side(step, lambda: [kc.clone(), vc.clone()])


def test_layer_forms_refuse_other_sizes():
    x, p = layer()
    stats, o = torch.empty((2, 4, 200, 2), device="cuda"), torch.empty(x.shape, device="cuda",
                                                                      dtype=torch.float16)
    dz = torch.empty(x.shape, device="cuda")
    for name in ("ln1", "W_Q", "W_O", "W_1", "b_1", "W_2", "b_2"):
        bad = dict(p)
        bad[name] = p[name][:-1].contiguous()
        with pytest.raises(ValueError):
            bpt.layer_forward_window(x, bad, 4, 64)
        with pytest.raises(ValueError):
            bpt.layer_backward_window(x, bad, 4, 64, 0, stats, o, dz)
    host = torch.empty(1 << 24, dtype=torch.uint8)
    with pytest.raises(ValueError):
        bpt.layer_forward_window(x, p, 4, 64, workspace=host)
    with pytest.raises(ValueError):
        bpt.layer_backward_window(x, p, 4, 64, 0, stats, o, dz, workspace=host)


def test_a_row_of_nothing_but_nan_stays_so():
    """V is NaN throughout, Q and K are finite: every visible row is NaN, and
    the rows past a length are 0 all the same."""
    q, k = tensors(9, (1, 700, 2, 64), (1, 700, 2, 64))
    lens = torch.tensor([650], dtype=torch.int32, device="cuda")
    out = bpt.attn_window_forward(q, k, torch.full_like(k, float("nan")), 400, 3, lens=lens)
    assert torch.isnan(out[:, :650]).all() and (out[:, 650:] == 0).all()
    v = torch.zeros_like(k)
    v[:, 100, :, 7] = float("nan")
    out = bpt.attn_window_forward(q, k, v, 400, 3, lens=lens)
    bad = torch.isnan(out)
    assert bad[:, 100:500, :, 7].all()
    bad[:, 100:500, :, 7] = False
    assert not bad.any()


@pytest.mark.parametrize("captured", [False, True])
def test_gradients_one_after_another_through_one_workspace(captured):
    """The launches of a call overlap; those of the next call, and whatever
    reads the gradients, find all of them done: bitwise what each call gives
    alone."""
    calls = []
    for i, (B, n, h, hkv, dk, window, sinks, dt) in enumerate([
            (3, 700, 4, 2, 64, 100, 4, BF), (1, 2100, 4, 1, 128, 300, 130, torch.float16),
            (2, 60, 2, 2, 64, 64, 0, torch.float16), (1, 1500, 2, 2, 128, 1500, 0, BF)]):
        q, do = tensors(20 + i, (B, n, h, dk), (B, n, h, dk), dt=dt)
        k, v = tensors(30 + i, (B, n, hkv, dk), (B, n, hkv, dk), dt=dt)
        lens = torch.tensor([n - 37 * b for b in range(B)], dtype=torch.int32, device="cuda")
        stats = torch.empty((B, h, n, 2), device="cuda")
        o = bpt.attn_window_forward(q, k, v, window, sinks, lens=lens, stats=stats)
        want = bpt.attn_window_backward(q, k, v, o, stats, do, window, sinks, lens=lens)
        torch.cuda.synchronize()
        calls.append(((q, k, v, o, stats, do, window, sinks, lens), want))
    ws = max((bpt.attn_window_backward_workspace(a[0], a[1], a[6], a[7]) for a, _ in calls),
             key=torch.Tensor.numel)
    grads = [[torch.empty_like(w) for w in want] for _, want in calls]
    copies = [[torch.empty_like(w) for w in want] for _, want in calls]

    def every():
        for (args, _), into, copy in zip(calls, grads, copies):
            bpt.attn_window_backward(*args, into, ws)
            for c, g in zip(copy, into):
                c.copy_(g)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            every()
    for _ in range(10):
        for c in sum(copies, []):
            c.zero_()
        graph.replay() if captured else every()
        for (_, want), copy in zip(calls, copies):
            for w, c in zip(want, copy):
                assert torch.equal(w, c)

"""The layer with sliding-window attention (forward, gradients) and with a
paged cache (prefill, one-token steps) against an fp64 layer with autograd."""
import math

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from blockwise_attn_ffn_b200.inputs import LayerShape, make_inputs
from gpu_util import TOL_BF16
from oracle.attention import window_mask

pytestmark = pytest.mark.gpu
SHAPES = {
    64: LayerShape("win64", B=3, N=300, d=256, h=4, d_ff=512, causal=True, dtype="bf16", block=128,
                   seed=51, ln_scale=0.1, bias_scale=0.2),
    128: LayerShape("win128", B=2, N=413, d=256, h=2, d_ff=512, causal=True, dtype="bf16",
                    block=128, seed=52, ln_scale=0.1, bias_scale=0.2),
}


def layer64(inp, h, window, sinks, lens=None):
    """The layer in fp64 torch; returns (Z, leaves by name)."""
    t = {k: torch.tensor(np.asarray(inp[k], np.float64), device="cuda", requires_grad=True)
         for k in ("x", "gamma1", "beta1", "W_Q", "W_K", "W_V", "W_O", "gamma2", "beta2", "W_1",
                   "b_1", "W_2", "b_2")}
    x = t["x"]
    B, N, d = x.shape
    dk = d // h
    ln = lambda v, g, b: torch.nn.functional.layer_norm(v, (d,), g, b, 1e-5)
    u = ln(x, t["gamma1"], t["beta1"])
    q, k, v = ((u @ t[n]).view(B, N, h, dk) for n in ("W_Q", "W_K", "W_V"))
    ok = torch.stack([window_mask(N, N, window, sinks, N if lens is None else lens[b], "cuda")
                      for b in range(B)])
    s = torch.einsum("bihc,bjhc->bhij", q, k) / math.sqrt(dk)
    p = torch.softmax(s.masked_fill(~ok[:, None], -1e300), -1) * ok[:, None]
    o = torch.einsum("bhij,bjhc->bihc", p, v).reshape(B, N, d)
    y = x + o @ t["W_O"]
    f = torch.nn.functional.gelu(ln(y, t["gamma2"], t["beta2"]) @ t["W_1"] + t["b_1"])
    return y + f @ t["W_2"] + t["b_2"], t


def close(got, want):
    e = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert e.max() <= TOL_BF16[0] and e.mean() <= TOL_BF16[1], (e.max().item(), e.mean().item())


def no_fault(ws):
    st, site = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_OK, (bpt.status_string(st), site)


@pytest.mark.parametrize("dk,window,sinks,ragged", [(64, 100, 4, False), (64, 37, 0, True),
                                                    (128, 128, 130, True), (128, 1000, 0, False)])
def test_layer_forward_and_gradients(dk, window, sinks, ragged):
    cfg = SHAPES[dk]
    inp = make_inputs(cfg)
    dev = bpt.to_device(inp, "bf16")
    lens = [cfg.N - 57 * b for b in range(cfg.B)] if ragged else None
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    B, N, d, h = cfg.B, cfg.N, cfg.d, cfg.h
    stats = torch.empty((B, h, N, 2), device="cuda")
    o = torch.empty((B, N, d), dtype=torch.float16, device="cuda")
    out, ws = bpt.layer_forward_window(dev["x"], dev, h, window, sinks, lens=lt, stats=stats,
                                       keep_o=o)
    no_fault(ws)
    Z, t = layer64(inp, h, window, sinks, lens)
    close(out, Z.detach())
    plain, _ = bpt.layer_forward_window(dev["x"], dev, h, window, sinks, lens=lt)
    assert torch.equal(plain, out)
    g = torch.Generator(device="cuda").manual_seed(5)
    dZ = torch.randn((B, N, d), generator=g, device="cuda")
    grads, bws = bpt.layer_backward_window(dev["x"], dev, h, window, sinks, stats, o, dZ, lens=lt)
    no_fault(bws)
    Z.backward(dZ.double())
    want = {k: t[k].grad for k in ("x", "W_Q", "W_K", "W_V", "W_O", "W_1", "b_1", "W_2", "b_2")}
    want["ln1"] = torch.stack([t["gamma1"].grad, t["beta1"].grad])
    want["ln2"] = torch.stack([t["gamma2"].grad, t["beta2"].grad])
    for k, w in want.items():
        rel = ((grads[k].double() - w).norm() / w.norm()).item()
        assert rel <= 1e-2, (k, rel)


def test_a_window_of_everything_is_the_causal_layer():
    """window >= N: the plain causal layer's output up to the order of sums."""
    cfg = SHAPES[128]
    inp = make_inputs(cfg)
    dev = bpt.to_device(inp, "bf16")
    a, _ = bpt.layer_forward(dev["x"], dev, cfg.h, True)
    b, _ = bpt.layer_forward_window(dev["x"], dev, cfg.h, cfg.N)
    assert (a - b).abs().max() <= 2 * TOL_BF16[0] and (a - b).abs().mean() <= TOL_BF16[1]


@pytest.mark.parametrize("dk,window,sinks", [(64, 0, 0), (128, 60, 3)])
def test_prefill_then_steps_follow_the_whole_sequence(dk, window, sinks):
    """A padded batch of prompts into a cache, then one token at a time: every
    step's output is the whole sequence's at that position."""
    cfg = SHAPES[dk]
    inp = make_inputs(cfg)
    dev = bpt.to_device(inp, "bf16")
    B, N, d, h = cfg.B, cfg.N, cfg.d, cfg.h
    prompt = [N - 20 - 31 * b for b in range(B)]
    w = window or N
    want = layer64(inp, h, w, sinks)[0].detach()
    ps, per = 16, -(-N // 16)
    g = torch.Generator(device="cuda").manual_seed(7)
    total = B * per + 2
    table = torch.randperm(total, generator=g, device="cuda")[:B * per].view(B, per).int()
    kc = torch.full((total, h, ps, dk), math.nan, dtype=torch.float16, device="cuda")
    vc = kc.clone()
    acc = torch.full((B, h, per * ps), 5.0, device="cuda")
    pos = torch.zeros((B, h, per * ps), dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    counts = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    new = torch.empty_like(lens)
    out, ws = bpt.layer_forward_window(dev["x"], dev, h, w, sinks, lens=counts,
                                       cache=(kc, vc, table, lens), new_lens=new, acc=acc, pos=pos)
    no_fault(ws)
    assert new.tolist() == prompt
    for b in range(B):
        close(out[b, :prompt[b]], want[b, :prompt[b]])
    lens, new = new, lens
    dws = bpt.layer_decode_workspace(dev, kc, table, with_acc=True)
    for step in range(20):
        at = torch.tensor([n + step for n in prompt], device="cuda")
        x = dev["x"][torch.arange(B, device="cuda"), at].contiguous()
        z, _ = bpt.layer_decode(x, dev, kc, vc, table, lens, dws, window, sinks, acc=acc, pos=pos,
                                new_lens=new)
        close(z, want[torch.arange(B, device="cuda"), at])
        lens, new = new, lens
        assert lens.tolist() == [n + step + 1 for n in prompt]
    no_fault(dws)
    for b in range(B):
        n = prompt[b] + 20
        assert pos[b, 0, :n].tolist() == list(range(n))
        # 20 steps of weights that sum to one per head, spread over the slots
        assert (acc[b, :, :n].double().sum(-1) - 20).abs().max() < 20 * 1e-4
        assert (acc[b, :, n:] == 5.0).all()


def test_a_captured_step_replays():
    cfg = SHAPES[64]
    inp = make_inputs(cfg)
    dev = bpt.to_device(inp, "bf16")
    B, d, h, dk, ps = cfg.B, cfg.d, cfg.h, 64, 32
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    g = torch.Generator(device="cuda").manual_seed(9)
    kc = torch.randn((B * 4, h, ps, dk), generator=g, device="cuda").half()
    vc = torch.randn((B * 4, h, ps, dk), generator=g, device="cuda").half()
    lens = torch.tensor([5, 64, 100], dtype=torch.int32, device="cuda")
    new = torch.zeros_like(lens)
    ws = bpt.layer_decode_workspace(dev, kc, table)
    x = dev["x"][:, 0].contiguous()
    out = torch.empty((B, d), device="cuda")
    step = lambda: bpt.layer_decode(x, dev, kc, vc, table, lens, ws, new_lens=new, out=out)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, 3):
        x.copy_(dev["x"][:, i])
        lens.copy_(new)
        out.zero_()
        graph.replay()
        got, k1 = out.clone(), kc.clone()
        step()
        assert torch.equal(got, out) and torch.equal(k1, kc)
        assert new.tolist() == [n + i + 1 for n in (5, 64, 100)]
    no_fault(ws)

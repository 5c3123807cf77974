"""The paged key-value cache on the GPU: append, one-token attention and
eviction against fp64 definitions (oracle/attention.py), alone and together."""
import math

import pytest
import torch

import blockwise_attn_ffn_b200 as bpt
from oracle.attention import decode_attention, evict_order, visible_slots

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)


class Pool:
    """A cache whose pages lie in any order; table entries past a sequence's
    last page name no page at all."""

    def __init__(self, seed, lens, hkv, dk, ps, dt, room=0, per=None):
        g = gen(seed)
        self.B, self.hkv, self.dk, self.ps, self.dt = len(lens), hkv, dk, ps, dt
        self.n = list(lens)
        per = per or max(1, -(-(max(lens) + room) // ps))
        self.cap = per * ps
        used = [-(-(n + room) // ps) for n in lens]
        total = sum(used) + 2
        order = torch.randperm(total, generator=g, device="cuda").tolist()
        table = torch.full((self.B, per), -7, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            for i in range(min(u, per)):
                table[b, i] = order[at]
                at += 1
        self.table = table.cuda()
        self.k = randn(g, (total, hkv, ps, dk), dt)
        self.v = randn(g, (total, hkv, ps, dk), dt)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def rows(self, x, b, slots):
        """fp64 rows [len(slots), hkv, dk] of sequence b."""
        if not len(slots):
            return torch.zeros((0, self.hkv, self.dk), dtype=torch.float64, device="cuda")
        s = torch.tensor(list(slots), device="cuda")
        page = self.table[b].long()[s // self.ps]
        return x[page, :, s % self.ps].double()

    def poison(self, slots_of):
        """NaN and infinities wherever no visible slot lies."""
        keep = torch.zeros(self.k.shape[0], self.ps, dtype=torch.bool, device="cuda")
        for b in range(self.B):
            s = torch.tensor(slots_of(b), dtype=torch.long, device="cuda")
            if len(s):
                keep[self.table[b].long()[s // self.ps], s % self.ps] = True
        bad = ~keep[:, None, :, None].expand_as(self.k)
        self.k[bad] = math.nan
        self.v[bad] = math.inf


def no_fault(ws):
    st, site = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_OK, (bpt.status_string(st), site)


def decode_bounds(q, k, n, dt):
    """(u, c): half a step of the type, and the relative error that fp32 leaves
    in the weights: a score is a sum of dk products (at most 2 dk 2^-24 of the
    absolute products' sum, also where the tensor core truncates), it moves a
    weight and the sum of the weights; exp2 is good to 2^-21; the sums over n
    keys add n 2^-23 at most."""
    u = torch.finfo(dt).eps / 2
    dk = q.shape[-1]
    if n == 0:
        return u, 0.0
    g = q.shape[0] // k.shape[1]
    s_abs = torch.einsum("hd,jhd->hj", q.abs(), k.abs().repeat_interleave(g, 1)).max().item()
    s_abs /= math.sqrt(dk)
    return u, 2 * (2 * dk * 2.0 ** -24 * s_abs) + 2.0 ** -20 + n * 2.0 ** -23


CASES = [
    # lens, h, hkv, dk, ps, window, sinks, dtype, acc
    ([1], 1, 1, 64, 16, 0, 0, "bf16", False),
    ([0, 1, 5], 4, 2, 128, 16, 0, 0, "f16", True),
    ([63, 64, 65, 0, 129], 6, 2, 64, 5, 0, 0, "bf16", True),
    ([301], 12, 12, 64, 16, 0, 0, "bf16", False),
    ([1000, 17, 2500], 32, 2, 128, 48, 0, 0, "f16", True),     # 16 heads share one
    ([700, 90], 40, 2, 128, 16, 0, 0, "bf16", True),           # 20 heads: two chunks
    ([700, 90, 3], 8, 8, 128, 64, 100, 4, "f16", True),
    ([2049, 130, 40], 12, 4, 64, 32, 33, 70, "bf16", True),    # more sinks than some have
    ([5000], 8, 1, 128, 128, 1, 0, "bf16", True),              # only itself
    ([30011], 4, 4, 64, 64, 0, 0, "f16", True),
    ([200] * 300, 2, 1, 64, 16, 0, 0, "f16", False),           # more pairs than blocks
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[1:8])))
def test_decode_against_the_definition(case):
    lens, h, hkv, dk, ps, window, sinks, dt, with_acc = case
    dt = DT[dt]
    pool = Pool(1, lens, hkv, dk, ps, dt)
    pool.poison(lambda b: visible_slots(lens[b], window, sinks))
    g = gen(2)
    q = randn(g, (len(lens), h, dk), dt, 1.5)
    acc = torch.rand((len(lens), hkv, pool.cap), generator=g, device="cuda") if with_acc else None
    acc_out = torch.full_like(acc, -3.0) if with_acc else None
    ws = bpt.attn_decode_workspace(q, pool.k, pool.table, with_acc)
    out = torch.full_like(q, math.nan)
    bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens, window, sinks, acc=acc,
                    acc_out=acc_out, out=out, ws=ws)
    no_fault(ws)
    for b in list(range(len(lens)))[:12]:
        vis = visible_slots(lens[b], window, sinks)
        k, v = pool.rows(pool.k, b, vis), pool.rows(pool.v, b, vis)
        o, p, A = decode_attention(q[b].double(), k, v)
        u, c = decode_bounds(q[b].double(), k, len(vis), dt)
        # P is rounded once, the output once
        err = (out[b].double() - o).abs()
        assert (err <= (u + c) * A * (1 + u) + u * o.abs() + 1e-30 + 2.0 ** -25).all(), \
            (b, err.max().item())
        if with_acc:
            want = acc[b].double().clone()
            w = torch.zeros((hkv, pool.cap), dtype=torch.float64, device="cuda")
            if vis:
                w[:, vis] = p.view(hkv, h // hkv, -1).sum(1)
            want += w
            e = (acc_out[b].double() - want).abs()[:, :lens[b]]
            assert (e <= (c * w + (h // hkv + 1) * 2.0 ** -24 * want)[:, :lens[b]]).all()
            assert (acc_out[b, :, lens[b]:] == -3.0).all()


def test_decode_strides_streams_and_repeats():
    """q inside a packed projection, out inside a wider row, another stream,
    acc in place: bitwise what the plain call gives."""
    lens = [700, 3, 0, 260]
    pool = Pool(3, lens, 4, 128, 16, torch.bfloat16)
    g = gen(4)
    packed = randn(g, (4, 3, 8, 128), torch.bfloat16)
    q = packed[:, 1]
    acc = torch.rand((4, 4, pool.cap), generator=g, device="cuda")
    a = bpt.attn_decode(q.contiguous(), pool.k, pool.v, pool.table, pool.lens, 128, 4, acc=acc,
                        acc_out=(acc_a := acc.clone()))
    wide = torch.full((4, 8, 160), 5.0, dtype=torch.bfloat16, device="cuda")
    acc_b = acc.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = bpt.attn_decode_workspace(q, pool.k, pool.table, True)
    torch.cuda.synchronize()
    bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens, 128, 4, acc=acc_b,
                    out=wide[..., :128], ws=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(wide[..., :128], a) and (wide[..., 128:] == 5.0).all()
    assert torch.equal(acc_b, acc_a)


def test_one_workspace_serves_sizes_and_operators_in_turn():
    """Calls of different batches, heads and lengths, an append and an eviction
    through one workspace: each gives what it gives with its own."""
    cases = [([2000], 8, 1, 128, True), ([700, 90, 3] * 20, 8, 8, 64, False),
             ([5000, 1], 4, 4, 128, True), ([300] * 70, 2, 1, 64, False)]
    made = []
    for i, (lens, h, hkv, dk, with_acc) in enumerate(cases):
        pool = Pool(40 + i, lens, hkv, dk, 16, torch.bfloat16)
        q = randn(gen(50 + i), (len(lens), h, dk), torch.bfloat16)
        acc = torch.zeros((len(lens), hkv, pool.cap), device="cuda") if with_acc else None
        size = bpt.attn_decode_workspace(q, pool.k, pool.table, with_acc).numel()
        size = max(size, bpt.cache_workspace(pool.k, pool.table).numel())
        made.append((pool, q, acc, size))
    ws = torch.randint(0, 255, (max(m[3] for m in made),), dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    for turn in range(2):
        for pool, q, acc, _ in made:
            run = lambda w: bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens, acc=acc,
                                            acc_out=None if acc is None else acc.clone(), ws=w)
            assert torch.equal(run(ws), run(None))
            a, p, seen = evict_inputs(pool, 60, False)
            bpt.cache_evict(pool.k, pool.v, pool.table, pool.lens, a, p, seen, max(pool.n), ws=ws)
    no_fault(ws)


def test_decode_in_a_graph_follows_the_lengths():
    lens = [100, 400]
    pool = Pool(5, [500, 500], 2, 64, 16, torch.float16)
    pool.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    q = randn(gen(6), (2, 4, 64), torch.float16)
    ws = bpt.attn_decode_workspace(q, pool.k, pool.table)
    out = torch.empty_like(q)
    call = lambda: bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens, out=out, ws=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([1, 500], [499, 0], [64, 65]):
        pool.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(9.0)
        graph.replay()
        got = out.clone()
        call()
        assert torch.equal(got, out)
        assert (out[lens.index(0)] == 0).all() if 0 in lens else True
    no_fault(ws)


def test_a_page_outside_the_pool_is_reported_and_skipped():
    lens = [40, 40]
    pool = Pool(7, lens, 2, 64, 16, torch.float16)
    q = randn(gen(8), (2, 2, 64), torch.float16)
    good = bpt.attn_decode(q, pool.k, pool.v, pool.table, pool.lens)
    table = pool.table.clone()
    table[1, 1] = pool.k.shape[0]
    ws = bpt.attn_decode_workspace(q, pool.k, table)
    out = bpt.attn_decode(q, pool.k, pool.v, table, pool.lens, ws=ws)
    st, site = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_ERR_INDEX and site != 0
    assert torch.equal(out[0], good[0]) and torch.isfinite(out).all()
    no_fault(ws)  # read once, cleared
    # lengths outside the table: taken as the nearest
    lens2 = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    full = Pool(7, [48, 48], 2, 64, 16, torch.float16)
    out = bpt.attn_decode(q, full.k, full.v, full.table, lens2, ws=ws)
    st, _ = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_ERR_INDEX
    want = bpt.attn_decode(q, full.k, full.v, full.table, full.lens)
    assert (out[0] == 0).all() and torch.equal(out[1], want[1])


@pytest.mark.parametrize("lens,T,counts,hkv,dk,ps,dt,packed", [
    ([0], 1, None, 1, 64, 16, "bf16", False),
    ([5, 0, 64], 1, None, 8, 128, 16, "f16", True),
    ([5, 0, 64], 77, [77, 0, 13], 3, 64, 5, "bf16", True),
    ([15, 100], 1000, [999, 1000], 16, 128, 48, "f16", False),
    ([3, 9], 0, None, 2, 64, 16, "bf16", False),
], ids=str)
def test_append_writes_its_slots_and_no_others(lens, T, counts, hkv, dk, ps, dt, packed):
    dt, B = DT[dt], len(lens)
    pool = Pool(11, lens, hkv, dk, ps, dt, room=T)
    g = gen(12)
    if packed:
        kv = randn(g, (B, T, 2, hkv, dk), dt)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = randn(g, (B, T, hkv, dk), dt), randn(g, (B, T, hkv, dk), dt)
    acc = torch.rand((B, hkv, pool.cap), generator=g, device="cuda")
    pos = torch.randint(0, 99, (B, hkv, pool.cap), generator=g, device="cuda", dtype=torch.int32)
    seen = torch.tensor([n + 3 for n in lens], dtype=torch.int32, device="cuda")
    want = [x.clone() for x in (pool.k, pool.v, acc, pos)]
    cnt = counts or [T] * B
    for b in range(B):
        for t in range(cnt[b]):
            s = lens[b] + t
            page = int(pool.table[b, s // ps])
            want[0][page, :, s % ps] = k[b, t]
            want[1][page, :, s % ps] = v[b, t]
            want[2][b, :, s] = 0
            want[3][b, :, s] = lens[b] + 3 + t
    ws = bpt.cache_workspace(pool.k, pool.table)
    c = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    new = bpt.cache_append(k, v, pool.k, pool.v, pool.table, pool.lens, counts=c, acc=acc, pos=pos,
                           seen=seen, ws=ws)
    no_fault(ws)
    for got, w in zip((pool.k, pool.v, acc, pos), want):
        assert torch.equal(got, w)
    assert new.tolist() == [n + c for n, c in zip(lens, cnt)] and pool.lens.tolist() == lens


def test_append_without_room_drops_the_rest():
    pool = Pool(13, [14, 2], 2, 64, 16, torch.float16, per=1)
    k = randn(gen(14), (2, 5, 2, 64), torch.float16)
    before = pool.k.clone()
    ws = bpt.cache_workspace(pool.k, pool.table)
    new = bpt.cache_append(k, k, pool.k, pool.v, pool.table, pool.lens, ws=ws)
    st, _ = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_ERR_INDEX and new.tolist() == [16, 7]
    p0, p1 = int(pool.table[0, 0]), int(pool.table[1, 0])
    before[p0, :, 14:16] = k[0, :2].transpose(0, 1)
    before[p1, :, 2:7] = k[1].transpose(0, 1)
    assert torch.equal(pool.k, before)


def evict_inputs(pool, seed, ties):
    g = gen(seed)
    shape = (pool.B, pool.hkv, pool.cap)
    acc = torch.randn(shape, generator=g, device="cuda").mul(2).exp()
    if ties:
        acc = torch.randint(0, 4, shape, generator=g, device="cuda").float() / 4
        acc[..., ::7] = -0.0
    pos = torch.rand(shape, generator=g, device="cuda").argsort(-1).to(torch.int32) * 2
    seen = torch.full((pool.B,), 2 * pool.cap, dtype=torch.int32, device="cuda")
    return acc, pos, seen


def check_evicted(pool, before, acc, pos, seen, budget, recent, sinks, got, tail):
    k0, v0 = before
    acc_o, pos_o, new = got
    assert new.tolist() == [min(n, budget) for n in pool.n]
    kw, vw = k0.clone(), v0.clone()
    for b in range(pool.B):
        n = pool.n[b]
        for t in range(pool.hkv):
            a, p = acc[b, t, :n], pos[b, t, :n]
            order = evict_order(a.tolist(), p.tolist(), int(seen[b]), budget, recent, sinks)
            idx = torch.tensor(order, dtype=torch.long, device="cuda")
            m = len(order)
            assert torch.equal(acc_o[b, t, :m].view(torch.int32), a[idx].view(torch.int32))
            assert torch.equal(pos_o[b, t, :m], p[idx])
            assert torch.equal(acc_o[b, t, m:].view(torch.int32),
                               tail[0][b, t, m:].view(torch.int32))  # bits: NaN among them
            assert torch.equal(pos_o[b, t, m:], tail[1][b, t, m:])
            to = torch.arange(m, device="cuda")
            tab = pool.table[b].long()
            for w, src in ((kw, k0), (vw, v0)):
                w[tab[to // pool.ps], t, to % pool.ps] = src[tab[idx // pool.ps], t, idx % pool.ps]
    assert torch.equal(pool.k, kw) and torch.equal(pool.v, vw)


@pytest.mark.parametrize("lens,hkv,dk,ps,budget,recent,sinks,dt,ties", [
    ([1, 0, 9], 2, 64, 16, 4, 1, 1, "bf16", False),
    ([100, 37, 64, 0], 3, 128, 5, 36, 10, 4, "f16", True),
    ([1300, 1024, 1025], 2, 64, 16, 1024, 256, 4, "bf16", False),
    ([3000, 2999], 1, 64, 48, 1, 0, 0, "f16", True),
    ([5000, 4100], 2, 128, 64, 1000, 0, 0, "bf16", True),
    ([600], 2, 64, 16, 500, 600, 0, "f16", False),            # more protected than the budget
    ([40, 20], 2, 64, 16, 400, 5, 1, "bf16", False),          # nothing to do
    ([9001, 7000], 1, 64, 48, 3000, 100, 4, "f16", False),    # two, four and eight blocks per pair
    ([15000, 5], 1, 64, 64, 7600, 0, 0, "bf16", True),
    ([140001], 1, 64, 128, 20011, 500, 4, "f16", True),       # keys past the shared memory
], ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_keeps_what_the_definition_keeps(lens, hkv, dk, ps, budget, recent, sinks, dt, ties,
                                               in_place):
    pool = Pool(21, lens, hkv, dk, ps, DT[dt])
    acc, pos, seen = evict_inputs(pool, 22, ties)
    if ties and lens[0] > 50:
        acc[0, 0, 3], acc[0, 0, 40] = math.nan, math.inf
    before = (pool.k.clone(), pool.v.clone())
    ws = bpt.cache_workspace(pool.k, pool.table)
    a0, p0 = acc.clone(), pos.clone()
    if in_place:
        lens_t = pool.lens.clone()
        new = bpt.cache_evict(pool.k, pool.v, pool.table, lens_t, acc, pos, seen, budget, recent,
                              sinks, ws=ws)
        assert new is lens_t
        got, tail = (acc, pos, new), (a0, p0)
    else:
        tail = (torch.full_like(acc, -1.0), torch.full_like(pos, -1))
        got = (tail[0].clone(), tail[1].clone(), torch.zeros_like(pool.lens))
        bpt.cache_evict(pool.k, pool.v, pool.table, pool.lens, acc, pos, seen, budget, recent,
                        sinks, acc_out=got[0], pos_out=got[1], new_lens=got[2], ws=ws)
        assert torch.equal(acc.view(torch.int32), a0.view(torch.int32))
    no_fault(ws)
    check_evicted(pool, before, a0, p0, seen, budget, recent, sinks, got, tail)


def test_evict_over_a_bad_page_reports_and_moves_the_rest():
    pool = Pool(23, [64], 1, 64, 16, torch.float16)
    acc, pos, seen = evict_inputs(pool, 24, False)
    table = pool.table.clone()
    table[0, 3] = -1
    ws = bpt.cache_workspace(pool.k, table)
    k0 = pool.k.clone()
    bpt.cache_evict(pool.k, pool.v, table, pool.lens, acc, pos, seen, 16, ws=ws)
    st, _ = bpt.bpt_read_device_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == bpt.BPT_ERR_INDEX
    other = [p for p in range(k0.shape[0]) if p != int(table[0, 0])]
    assert torch.equal(pool.k[other], k0[other])  # only the first page changed


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_decoding_with_eviction_step_by_step(dt):
    """A prompt, then tokens one by one: append, attend with weights gathered,
    evict when over the budget; the state follows the definition's."""
    dt = DT[dt]
    B, h, hkv, dk, ps, budget = 3, 6, 2, 64, 16, 40
    prompt = [30, 1, 41]
    pool = Pool(31, [0, 0, 0], hkv, dk, ps, dt, room=64)
    g = gen(32)
    acc = torch.zeros((B, hkv, pool.cap), device="cuda")
    pos = torch.zeros((B, hkv, pool.cap), dtype=torch.int32, device="cuda")
    seen = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws_c = bpt.cache_workspace(pool.k, pool.table)
    ws_d = bpt.attn_decode_workspace(torch.empty(B, h, dk, dtype=dt), pool.k, pool.table, True)
    lens, new = pool.lens, torch.empty_like(pool.lens)
    # the definition's state: per sequence and head, lists of (k, v, weight, position)
    state = [[[] for _ in range(hkv)] for _ in range(B)]
    for step in range(30):
        T = max(prompt) if step == 0 else 1
        cnt = prompt if step == 0 else [1] * B
        k, v = randn(g, (B, T, hkv, dk), dt), randn(g, (B, T, hkv, dk), dt)
        counts = torch.tensor(cnt, dtype=torch.int32, device="cuda")
        bpt.cache_append(k, v, pool.k, pool.v, pool.table, lens, counts=counts, new_lens=new,
                         acc=acc, pos=pos, seen=seen, ws=ws_c)
        lens, new = new, lens
        for b in range(B):
            for t in range(hkv):
                for i in range(cnt[b]):
                    state[b][t].append([k[b, i, t].double(), v[b, i, t].double(), 0.0,
                                        int(seen[b]) + i])
        seen += counts
        q = randn(g, (B, h, dk), dt)
        out = bpt.attn_decode(q, pool.k, pool.v, pool.table, lens, acc=acc, ws=ws_d)
        for b in range(B):
            n = len(state[b][0])
            kk = torch.stack([torch.stack([e[0] for e in state[b][t]]) for t in range(hkv)], 1)
            vv = torch.stack([torch.stack([e[1] for e in state[b][t]]) for t in range(hkv)], 1)
            o, p, A = decode_attention(q[b].double(), kk, vv)
            u, c = decode_bounds(q[b].double(), kk, n, dt)
            assert ((out[b].double() - o).abs() <= (u + c) * A * (1 + u) + u * o.abs()
                    + 2.0 ** -25).all(), step
            w = p.view(hkv, h // hkv, n).sum(1)
            a = acc[b].double().cpu()
            for t in range(hkv):
                for j, e in enumerate(state[b][t]):
                    e[2] += float(w[t, j])
                    assert abs(float(a[t, j]) - e[2]) <= (step + 1) * (c + 2.0 ** -22) * max(e[2], 1)
                    e[2] = float(a[t, j])  # ties and near ties follow the stored weight
        bpt.cache_evict(pool.k, pool.v, pool.table, lens, acc, pos, seen, budget, 8, 2, ws=ws_c)
        for b in range(B):
            for t in range(hkv):
                s = state[b][t]
                order = evict_order([e[2] for e in s], [e[3] for e in s], int(seen[b]), budget, 8, 2)
                state[b][t] = [s[i] for i in order]
                n = len(order)
                assert pos[b, t, :n].tolist() == [e[3] for e in state[b][t]]
        assert lens.tolist() == [len(state[b][0]) for b in range(B)]
    no_fault(ws_c)
    no_fault(ws_d)

"""The paged calls as programs arrange them: a whole decode step on a side stream, in a captured graph and in two
streams at once; caches whose keys, values and copies lie differently; strided arrays of every kind; very
many and very small requests."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """Append, attention, weights and eviction of 3 requests on buffers of its own."""

    def __init__(self, seed, stream=None):
        g = torch.Generator().manual_seed(seed)
        self.k = torch.randn(40, 16, 2, 64, generator=g).to(torch.bfloat16).cuda()
        self.v = torch.randn(40, 16, 2, 64, generator=g).to(torch.bfloat16).cuda()
        self.q = torch.randn(3, 8, 64, generator=g).to(torch.bfloat16).cuda()
        self.k_new = torch.randn(3, 2, 64, generator=g).to(torch.bfloat16).cuda()
        self.v_new = torch.randn(3, 2, 64, generator=g).to(torch.bfloat16).cuda()
        self.table = torch.randperm(24, generator=g).to(torch.int32).reshape(3, 8).cuda()
        self.new = (torch.arange(15, dtype=torch.int32) + 25).reshape(3, 5).cuda()
        self.lens, self.starts = i32([100, 17, 1]), i32([0, 1, 2, 3])
        self.logits, self.w = torch.zeros(3, 8, 128, device="cuda"), torch.zeros(3, 2, 128, device="cuda")
        self.stream = stream

    def run(self):
        kw = {} if self.stream is None else dict(stream=self.stream)
        dcp.dcp_kv_append(self.k_new, self.v_new, self.k, self.v, self.table, self.lens, self.starts, **kw)
        if self.stream is None:
            out, lse = dcp.paged_attention(self.q, self.k, self.v, self.table, self.lens, logits=self.logits)
            send = dcp.paged_attention_pack(self.q, self.k, self.v, self.table, self.lens, 8)
        else:
            out, lse = torch.empty_like(self.q), torch.empty(3, 8, device="cuda")
            send = torch.empty(8, 3, 1, 66, dtype=self.q.dtype, device="cuda")
            dcp.dcp_paged_attention(self.q, self.k, self.v, self.table, self.lens, out, lse, logits=self.logits, **kw)
            dcp.dcp_paged_attention_pack(self.q, self.k, self.v, self.table, self.lens, send, 8, **kw)
        dcp.dcp_kv_weights(self.logits, lse, self.lens, self.w, **kw)
        if self.stream is None:
            kept, lens, weights = dcp.kv_evict(self.w, self.k, self.v, self.table, self.lens, self.new, 70, 8)
        else:
            kept = torch.empty(3, 2, 70, dtype=torch.int32, device="cuda")
            lens, weights = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, 2, 128, device="cuda")
            dcp.dcp_kv_evict(self.w, self.k, self.v, self.table, self.lens, self.k, self.v, self.new, 70, 8, kept, lens,
                             weights, **kw)
        after, sums = dcp.paged_attention(self.q, self.k, self.v, self.new, lens) if self.stream is None else (out, lse)
        return [self.k, self.v, out, lse, send.view(torch.int16), self.logits, self.w, kept, lens, weights, after, sums]


def same(a, b, n=12):
    return all(torch.equal(x, y) for x, y in zip(a[:n], b[:n]))


def test_a_step_on_a_side_stream():
    """As the current stream, as an argument, and as a raw handle."""
    want = Step(1).run()
    s = torch.cuda.Stream()
    one, two, three = Step(1), Step(1, s), Step(1, s.cuda_stream)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = one.run()
    got2, got3 = two.run(), three.run()
    torch.cuda.synchronize()
    assert same(got, want) and same(got2, want, 10) and same(got3, want, 10)


def test_steps_of_two_streams_at_once():
    want = [Step(i).run() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        steps = [Step(i) for i in range(2)]
        torch.cuda.synchronize()
        got = []
        for st, s in zip(steps, streams):
            with torch.cuda.stream(s):
                got.append(st.run())
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


def test_a_step_in_two_graphs_replayed_in_turn():
    """Two graphs, each with a workspace and results of its own, replayed alternately and at the same time."""
    want = [Step(i).run() for i in range(2)]
    first = [Step(i) for i in range(2)]
    fresh = [(s.k.clone(), s.v.clone()) for s in first]
    graphs, outs = [], []
    for s in first:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, (k, v) in zip(first, fresh):
            s.k.copy_(k), s.v.copy_(v), s.w.zero_(), s.logits.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("width", [None, 700])
def test_keys_and_values_that_lie_differently(page, width):
    """Keys by slots, values by heads, out of a larger pool; the eviction's copies the other way round."""
    case = ref.PagedCase([70, 33, 0, 129], 3, 64, page, "bf16", seed=3, width=width)
    k, v, table = case.gpu()
    big = torch.full((case.pages + 2, 5, page, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[1:-1, 1:4, :, :64] = v.permute(0, 2, 1, 3)
    v = big[1:-1, 1:4, :, :64].permute(0, 2, 1, 3)
    q = torch.randn(4, 6, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out, lse = dcp.paged_attention(q.cuda(), k, v, table, i32(case.lens))
    r = ref.attention(q, case.keys, case.values, 0.125)
    ref.assert_attention(out, lse, r, 129, "bf16")
    w = torch.rand(4, 3, 129, generator=torch.Generator().manual_seed(4))
    new = torch.randperm(16, generator=torch.Generator().manual_seed(5)).to(torch.int32).reshape(4, 4).cuda()
    ko = torch.zeros(16, 3, 16, 64, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    vo = torch.zeros(16, 16, 3, 72, dtype=torch.bfloat16, device="cuda")[..., :64]
    kept, nl, nw = dcp.kv_evict(w.cuda(), k, v, table, i32(case.lens), new, 60, 7, k_out=ko, v_out=vo)
    for b, n in enumerate(case.lens):
        m = min(n, 60)
        assert int(nl[b]) == m
        for h in range(3):
            sel = ref.select(w[b, h, :n].numpy(), 60, 7)
            assert kept[b, h].tolist() == sel + [-1] * (60 - m)
            rows = torch.stack([ko[int(new[b, i // 16]), i % 16, h] for i in range(m)]) if m else ko[0, :0, 0]
            assert torch.equal(rows.cpu(), case.keys[b][sel, h])
            rows = torch.stack([vo[int(new[b, i // 16]), i % 16, h] for i in range(m)]) if m else vo[0, :0, 0]
            assert torch.equal(rows.cpu(), case.values[b][sel, h])


def test_strided_weights_logits_and_lse():
    """Every array of the weights and of the eviction a view of a larger one, the LSE a transposed one."""
    B, H, heads, cap = 3, 6, 2, 77
    lens = [77, 20, 0]
    logits = torch.randn(B, 2 * H, cap + 9, generator=torch.Generator().manual_seed(1)).cuda()[:, 1::2, 4:-5]
    lse = (torch.randn(H, B, generator=torch.Generator().manual_seed(2)) + 4).cuda().t()
    store = torch.full((heads, B, cap + 30), 7.0, device="cuda")
    w = store[:, :, 3:3 + cap + 10].permute(1, 0, 2)  # wider than the logits
    w.zero_()
    dcp.dcp_kv_weights(logits, lse, i32(lens), w)
    want = ref.weights(logits.cpu().numpy(), lse.cpu().numpy(), np.zeros((B, heads, cap + 10), np.float32), lens, True)
    # as in test_gpu_paged_cache.check_weights: exp's argument and own error, an addition per head
    assert (np.abs(w.cpu().double().numpy() - want) <= (2.0 ** -18 + 4 * 2.0 ** -24) * want).all()
    assert (store[:, :, :3] == 7).all() and (store[:, :, 3 + cap + 10:] == 7).all()
    k = torch.randn(B * 5, 16, heads, 16, device="cuda").to(torch.bfloat16)
    table = torch.arange(B * 5, dtype=torch.int32, device="cuda").reshape(B, 5)
    ko, vo = torch.zeros(B * 2, 16, heads, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(
        B * 2, 16, heads, 16, dtype=torch.bfloat16, device="cuda")
    tables = torch.full((B, 9), -1, dtype=torch.int32, device="cuda")
    tables[:, 3:5] = torch.arange(B * 2, dtype=torch.int32, device="cuda").reshape(B, 2)
    kept, nl = torch.empty(B, heads, 30, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    out = torch.full((heads, B, 50), 7.0, device="cuda")
    nw = out[:, :, 2:42].permute(1, 0, 2)
    dcp.dcp_kv_evict(w, k, k, table, i32(lens), ko, vo, tables[:, 3:5], 30, 3, kept, nl, nw)
    for b, n in enumerate(lens):
        for h in range(heads):
            sel = ref.select(w[b, h, :n].cpu().numpy(), 30, 3)
            assert kept[b, h].tolist() == sel + [-1] * (30 - len(sel))
            assert torch.equal(nw[b, h, :len(sel)], w[b, h, sel]) and (nw[b, h, len(sel):] == 0).all()
    assert (out[:, :, :2] == 7).all() and (out[:, :, 42:] == 7).all()
    assert torch.equal(ko, vo)


def test_logits_of_no_room_and_one_head_per_rank():
    case = ref.PagedCase([40, 9], 2, 64, 16, "bf16", seed=6)
    k, v, table = case.gpu()
    q = torch.randn(2, 64, 64, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()
    out, lse = dcp.paged_attention(q, k, v, table, i32(case.lens), logits=torch.empty(2, 64, 0, device="cuda"))
    r = ref.attention(q.cpu(), case.keys, case.values, 0.125)
    ref.assert_attention(out, lse, r, 40, "bf16")
    send = dcp.paged_attention_pack(q, k, v, table, i32(case.lens), 64)
    assert torch.equal(send.view(torch.int16), dcp.pack(out, lse, 64).view(torch.int16))


@pytest.mark.parametrize("B,H", [(100000, 1), (30000, 8)])
def test_very_many_requests(B, H):
    """Requests of 0 to 4 positions in pages of 4, against sums over the whole batch in 64 bits."""
    lens = torch.arange(B, device="cuda") % 5
    k = torch.randn(B, 4, 1, 64, device="cuda").to(torch.bfloat16)
    v, q = torch.randn_like(k), torch.randn(B, H, 64, device="cuda").to(torch.bfloat16)
    table = torch.randperm(B, device="cuda").to(torch.int32)[:, None]
    out, lse = dcp.paged_attention(q, k, v, table, lens.to(torch.int32))
    kk, vv = k[table[:, 0].long(), :, 0].double(), v[table[:, 0].long(), :, 0].double()
    x = torch.einsum("bhd,bpd->bhp", q.double(), kk) / 8
    x = torch.where(torch.arange(4, device="cuda") < lens[:, None, None], x, -math.inf)
    want_lse = x.logsumexp(-1)
    want = torch.einsum("bhp,bpd->bhd", torch.where(lens[:, None, None] > 0, (x - want_lse[..., None]).exp(), 0.0), vv)
    empty = lens == 0
    assert (out[empty] == 0).all() and (lse[empty] == -math.inf).all()
    # one rounding to bf16 of values below 8 in size, and fp32 arithmetic
    assert float((out.double() - want).abs().max()) <= 8 * 2.0 ** -9 + 1e-4
    assert float((lse[~empty].double() - want_lse[~empty]).abs().max()) <= 1e-5
    # append one token to each that has room, then look it up
    new = torch.randn(B, 1, 64, device="cuda").to(torch.bfloat16)
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    dcp.dcp_kv_append(new, new, k, v, table, (lens + 1).to(torch.int32), starts)
    room = lens < 4
    rows = k[table[:, 0].long(), lens.clamp(max=3), 0]
    assert torch.equal(rows[room], new[room, 0])
    assert torch.equal(v[table[:, 0].long()[room], lens[room], 0], new[room, 0])


def test_empty_calls_of_every_kind():
    k = torch.ones(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    none, table = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert dcp.paged_attention_pack(q, k, k, table, none, 2).shape == (2, 0, 2, 66)
    dcp.dcp_kv_weights(torch.zeros(0, 4, 8, device="cuda"), torch.zeros(0, 4, device="cuda"), none,
                       torch.zeros(0, 2, 8, device="cuda"))
    dcp.dcp_kv_weights(torch.zeros(1, 4, 0, device="cuda"), torch.zeros(1, 4, device="cuda"), i32([3]),
                       torch.zeros(1, 2, 5, device="cuda"))
    kept, nl, nw = dcp.kv_evict(torch.zeros(0, 2, 8, device="cuda"), k, k, table, none, table, 10, 2, k_out=k.clone(),
                                v_out=k.clone())
    assert kept.shape == (0, 2, 10) and nl.shape == (0,) and nw.shape == (0, 2, 10)
    # weights without room hold nothing to keep
    out = k.clone()
    kept, nl, nw = dcp.kv_evict(torch.zeros(1, 2, 0, device="cuda"), k, k, i32([[0, 1]]), i32([20]), i32([[0]]), 10, 2,
                                k_out=out, v_out=k.clone())
    assert (kept == -1).all() and nl.tolist() == [0] and (nw == 0).all() and torch.equal(out, k)

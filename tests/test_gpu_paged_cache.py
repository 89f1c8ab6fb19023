"""Append, accumulated weights and eviction against their definitions, and a decode loop of several
ranks that uses all of the paged calls together."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same_bits(a: torch.Tensor, b: torch.Tensor) -> bool:
    it = torch.int32 if a.element_size() == 4 else torch.int16
    return torch.equal(a.cpu().contiguous().view(it), b.cpu().contiguous().view(it))


# ---- append -------------------------------------------------------------------------------------
def append_ref(k, k_new, table, lens, starts, page, shard, n, s):
    """The pool after the append, by loops."""
    out = k.clone()
    for r in range(len(lens)):
        for t in range(max(0, starts[r]), min(starts[r + 1], k_new.shape[0])):
            pos = lens[r] - (starts[r + 1] - t)
            if pos < 0 or (pos // s) % n != shard:
                continue
            p = pos // (n * s) * s + pos % s
            if p // page >= table.shape[1]:
                continue
            pg = int(table[r, p // page])
            if 0 <= pg < k.shape[0]:
                out[pg, p % page] = k_new[t]
    return out


def check_append(lens, starts, T, heads, D, page, dtype, layout="slots", shard=0, n=1, s=1, width=None, seed=0,
                 fresh=None):
    wide = width if width is not None else max(1, max(-(-x // page) for x in lens))
    case = ref.PagedCase(lens, heads, D, page, dtype, layout, width=width, seed=seed, spare=len(lens) * wide)
    k, v, table = case.gpu()
    # every entry names a page of its own: the tables of requests that may grow (two tokens of one
    # call in the same slot would leave either's row)
    table_cpu = torch.arange(table.numel(), dtype=torch.int32).reshape(table.shape) if fresh is None else fresh
    g = torch.Generator().manual_seed(seed + 1)
    k_new = torch.randn(T, heads, D, generator=g).to(ref.DTYPES[dtype])
    v_new = torch.randn(T, heads, D, generator=g).to(ref.DTYPES[dtype])
    want_k = append_ref(k.cpu(), k_new, table_cpu, lens, starts, page, shard, n, s)
    want_v = append_ref(v.cpu(), v_new, table_cpu, lens, starts, page, shard, n, s)
    dcp.dcp_kv_append(k_new.cuda(), v_new.cuda(), k, v, table_cpu.cuda(), i32(lens), i32(starts), shard=shard,
                      num_shards=n, interleave=s)
    assert same_bits(k, want_k) and same_bits(v, want_v)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [8, 64, 80, 128, 256])
def test_append_decode_step(dtype, D):
    check_append([1, 16, 17, 40, 33], [0, 1, 2, 3, 4, 5], 5, 3, D, 16, dtype)


@pytest.mark.parametrize("layout", ["slots", "heads", "mixed"])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_append_prompts(layout, page):
    """Requests of 0 to 70 new tokens, padding tokens at the end, a token before the first request."""
    check_append([70, 9, 50, 33], [2, 72, 72, 85, 86], 90, 2, 64, page, "bf16", layout)


@pytest.mark.parametrize("n,s", [(2, 1), (4, 16), (3, 5), (64, 1), (2, 2 ** 31 - 1)])
def test_append_shards(n, s):
    for shard in sorted({0, 1, n - 1}):
        check_append([100, 1, 37], [0, 60, 61, 80], 80, 2, 64, 8, "bf16", shard=shard, n=n, s=s, width=20)


def test_append_skips_what_has_no_place():
    """Positions below 0 (more new tokens than the length), past the table, in pages outside the
    pool, negative lengths; nothing else changes (pools compared whole)."""
    table = torch.tensor([[0, -1, 2], [3, 1 << 30, 4], [5, 1, -2 ** 31]], dtype=torch.int32)
    check_append([48, 3, 60], [0, 48, 60, 120], 125, 2, 64, 16, "bf16", width=3, fresh=table)
    check_append([-5, 0, 48], [0, 2, 4, 6], 6, 2, 64, 16, "bf16", width=3, fresh=table)


def test_append_nothing():
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    new = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_append(new[:0], new[:0], k, k.clone(), torch.zeros(1, 2, dtype=torch.int32, device="cuda"), i32([4]),
                      i32([0, 0]))
    dcp.dcp_kv_append(new, new, k, k.clone(), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), i32([]), i32([0]))
    assert (k == 0).all()


def test_append_many_requests_and_strided_rows():
    R = 1500
    lens = [(r * 7) % 30 + 1 for r in range(R)]
    starts = list(range(R + 1))
    case = ref.PagedCase(lens, 1, 64, 16, "bf16", seed=3)
    k, v, table = case.gpu()
    qkv = torch.randn(R, 3, 64, device="cuda").to(torch.bfloat16)
    before = k.clone()
    dcp.dcp_kv_append(qkv[:, 1:2], qkv[:, 2:], k, v, table, i32(lens), i32(starts))
    for r in (0, 1, 700, R - 1):
        p = lens[r] - 1
        pg = int(case.table[r, p // 16])
        assert torch.equal(k[pg, p % 16, 0], qkv[r, 1]) and torch.equal(v[pg, p % 16, 0], qkv[r, 2])
        before[pg, p % 16, 0] = qkv[r, 1]
    want = append_ref(case.k, qkv[:, 1:2].cpu(), case.table, lens, starts, 16, 0, 1, 1)
    assert same_bits(k, want)


@pytest.mark.parametrize("heads", [33, 70])
def test_append_many_heads_and_tokens(heads):
    check_append([700, 3, 1400], [0, 700, 703, 1900], 1905, heads, 8, 16, "bf16", n=1)


def test_append_on_another_stream_and_in_a_graph():
    lens, T = [20, 33], 4
    case = ref.PagedCase(lens, 2, 64, 16, "bf16", seed=9)
    k, v, table = case.gpu()
    new = torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16)
    want = append_ref(case.k, new.cpu(), case.table, lens, [0, 1, 4], 16, 0, 1, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    seq, starts = i32(lens), i32([0, 1, 4])
    torch.cuda.synchronize()
    dcp.dcp_kv_append(new, new, k, v, table, seq, starts, stream=s)
    s.synchronize()
    assert same_bits(k, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dcp.dcp_kv_append(new, new, k, v, table, seq, starts)
    new.copy_(torch.randn_like(new))
    seq.copy_(torch.tensor([19, 30], dtype=torch.int32))
    graph.replay()
    want = append_ref(want, new.cpu(), case.table, [19, 30], [0, 1, 4], 16, 0, 1, 1)
    assert same_bits(k, want)


# ---- accumulated weights --------------------------------------------------------------------------
def check_weights(B, H, heads, cap, lens, base_e=True, lo_pad=0, w_pad=0, seq=None, offset=0, **kw):
    g = torch.Generator().manual_seed(B * 100 + H)
    logits = torch.full((B, H, cap + lo_pad), float("nan"))
    for b in range(B):
        logits[b, :, :lens[b]] = torch.randn(H, lens[b], generator=g) * 3
    lse = torch.randn(B, H, generator=g) + 4
    lse.view(-1)[1::5] = float("-inf")
    lse.view(-1)[3::7] = float("nan")
    if not base_e:
        lse = lse / math.log(2.0)
    w = torch.rand(B, heads, cap + w_pad, generator=g)
    store = Guarded((B, heads, cap + w_pad + offset), torch.float32)
    store.tensor.fill_(5.0)
    store.tensor[:, :, offset:] = w.cuda()
    dcp.dcp_kv_weights(logits.cuda(), lse.cuda(), i32(lens if seq is None else seq), store.tensor[:, :, offset:],
                       is_lse_base_on_e=base_e, **kw)
    store.check()
    assert (store.tensor[:, :, :offset] == 5.0).all()
    want = ref.weights(logits.numpy(), lse.numpy(), w.numpy(), lens, base_e)
    got = store.tensor[:, :, offset:].cpu().double().numpy()
    assert np.isfinite(got).all()
    # exp's argument: one rounding of x - l and one of a base change, each 2^-24 of their size
    # (below 32 here, so 2^-18 of the term in all, exp's own error with it); each of the G + 1
    # additions rounds once
    err = np.abs(got - want)
    added = want - w.double().numpy()
    assert (err <= 2.0 ** -18 * added + (H // heads + 1) * 2.0 ** -24 * want).all(), (err / np.maximum(added, 1e-30)).max()
    for b in range(B):
        assert np.array_equal(got[b, :, lens[b]:], w.double().numpy()[b, :, lens[b]:])


@pytest.mark.parametrize("H,heads", [(1, 1), (8, 2), (6, 6), (15, 3), (32, 2), (40, 1)])
@pytest.mark.parametrize("base_e", [True, False])
def test_weights(H, heads, base_e):
    check_weights(5, H, heads, 333, [0, 1, 64, 255, 333], base_e)


@pytest.mark.parametrize("lo_pad,w_pad,offset", [(0, 0, 0), (1, 0, 0), (3, 2, 1), (4, 8, 4), (0, 5, 2)])
def test_weights_strides(lo_pad, w_pad, offset):
    check_weights(3, 8, 2, 1032, [1032, 5, 1000], lo_pad=lo_pad, w_pad=w_pad, offset=offset)


def test_weights_shards_and_lengths_past_the_arrays():
    seq = [0, 10, 100, 900]
    check_weights(4, 4, 2, 300, [ref.local_len(x, 1, 3, 4) for x in seq], seq=seq, shard=1, num_shards=3, interleave=4)
    check_weights(3, 4, 2, 50, [50, 0, 50], seq=[1 << 30, -4, 51])


def test_weights_many_rows_and_graph():
    check_weights(300, 8, 8, 20, [b % 21 for b in range(300)])
    logits = torch.randn(2, 4, 64, device="cuda")
    lse, seq, w = torch.zeros(2, 4, device="cuda"), i32([64, 3]), torch.zeros(2, 2, 64, device="cuda")
    dcp.dcp_kv_weights(logits, lse, seq, w)
    one = w.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dcp.dcp_kv_weights(logits, lse, seq, w)
    graph.replay()
    graph.replay()
    want = (one + one) + one
    assert torch.equal(w, want)
    with pytest.raises(ValueError):
        dcp.dcp_kv_weights(logits, lse[:, :2], seq, w)
    with pytest.raises(ValueError):
        dcp.dcp_kv_weights(logits.half(), lse, seq, w)
    with pytest.raises(dcp.DCPError):
        dcp.dcp_kv_weights(logits, lse, seq, torch.zeros(2, 3, 64, device="cuda"))


# ---- eviction -------------------------------------------------------------------------------------
def check_evict(lens, heads, D, page, keep, recent, dtype="bf16", layout="slots", weights=None, new_page=None,
                cap=None, new_cap=None, seed=0, seq=None, same_pool=False, bad_src=(), bad_dst=(), **kw):
    case = ref.PagedCase(lens, heads, D, page, dtype, layout, seed=seed)
    B, n_max = len(lens), max(max(lens), 1)
    cap = n_max if cap is None else cap
    new_cap = max(cap, keep) if new_cap is None else new_cap
    g = torch.Generator().manual_seed(seed + 5)
    w = torch.randn(B, heads, cap, generator=g).exp() if weights is None else weights
    k, v, table = case.gpu()
    new_page = page if new_page is None else new_page
    width = -(-keep // new_page) + 1
    table_cpu = case.table.clone()
    for b, j in bad_src:
        table_cpu[b, j] = [-1, case.pages][j % 2]
    order = torch.randperm(B * width, generator=g).to(torch.int32).reshape(B, width)
    if same_pool:
        extra = torch.zeros(B * width, *k.shape[1:], dtype=k.dtype, device="cuda")
        k, v = torch.cat([k, extra]), torch.cat([v, extra])
        k_out, v_out, order = k, v, order + case.pages
    else:
        k_out = torch.zeros(B * width, new_page, heads, D, dtype=k.dtype, device="cuda")
        v_out = torch.zeros_like(k_out)
    for b, j in bad_dst:
        order[b, j] = -7
    before = k_out.clone(), v_out.clone()
    kept, nl = Guarded((B, heads, keep), torch.int32), Guarded((B,), torch.int32)
    nw = Guarded((B, heads, new_cap), torch.float32)
    dcp.dcp_kv_evict(w.cuda(), k, v, table_cpu.cuda(), i32(lens if seq is None else seq), k_out, v_out, order.cuda(),
                     keep, recent, kept.tensor, nl.tensor, nw.tensor, **kw)
    kept.check(), nl.check(), nw.check()
    want_k, want_v = before
    for b in range(B):
        n = min(lens[b], cap)
        m = min(n, keep)
        assert int(nl.tensor[b]) == m
        for h in range(heads):
            sel = ref.select(w[b, h, :n].numpy(), keep, recent)
            assert kept.tensor[b, h].tolist() == sel + [-1] * (keep - m), (b, h)
            row = torch.zeros(new_cap)
            row[:m] = w[b, h, sel]
            assert torch.equal(nw.tensor[b, h].cpu().view(torch.int32), row.view(torch.int32))
            for i, p in enumerate(sel):
                if (b, p // page) in bad_src or (b, i // new_page) in bad_dst:
                    continue
                pg = int(order[b, i // new_page])
                want_k[pg, i % new_page, h] = case.keys[b][p, h]
                want_v[pg, i % new_page, h] = case.values[b][p, h]
    assert same_bits(k_out, want_k) and same_bits(v_out, want_v)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp16", 96), ("fp32", 128), ("bf16", 256), ("bf16", 8)])
@pytest.mark.parametrize("recent", [0, 5, 40])
def test_evict(dtype, D, recent):
    check_evict([0, 1, 39, 40, 41, 100, 300], 2, D, 16, 40, recent, dtype)


@pytest.mark.parametrize("layout", ["slots", "heads", "mixed"])
@pytest.mark.parametrize("page,new_page", [(1, 3), (5, 16), (16, 16), (64, 8)])
def test_evict_pages(layout, page, new_page):
    check_evict([33, 200, 7], 3, 64, page, 30, 4, layout=layout, new_page=new_page)


@pytest.mark.parametrize("keep", [1, 2, 1023, 1024, 5000])
def test_evict_long(keep):
    check_evict([5000, 4999, 2600], 1, 64, 16, keep, keep // 4)


@pytest.mark.parametrize("n", [4096, 4097, 20011, 49152, 49153])
def test_evict_around_the_sizes_that_change_the_kernel(n):
    check_evict([n, n - 1], 1, 8, 64, n // 3, 17, seed=n)


def test_evict_long_rows_with_ties():
    g = torch.Generator().manual_seed(3)
    w = torch.randint(0, 3, (2, 1, 30000), generator=g).float()
    check_evict([30000, 29999], 1, 8, 64, 12000, 100, weights=w)
    w = torch.randint(0, 3, (1, 1, 60000), generator=g).float()
    check_evict([60000], 1, 8, 64, 25000, 0, weights=w)


def test_evict_on_another_stream_and_in_a_graph():
    case = ref.PagedCase([100, 30], 2, 64, 16, "bf16", seed=12)
    k, v, table = case.gpu()
    w = torch.rand(2, 2, 100, device="cuda")
    new = torch.arange(6, dtype=torch.int32, device="cuda").reshape(2, 3)
    ko, vo = torch.zeros(6, 16, 2, 64, dtype=k.dtype, device="cuda"), torch.zeros(6, 16, 2, 64, dtype=k.dtype, device="cuda")
    seq = i32([100, 30])
    want = dcp.kv_evict(w, k, v, table, seq, new, 40, 4, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    first = ko.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dcp.kv_evict(w, k, v, table, seq, new, 40, 4, k_out=ko, v_out=vo)
    ko.zero_()
    graph.replay()
    assert torch.equal(ko, first) and all(torch.equal(a, b) for a, b in zip(got, want))
    w.copy_(torch.rand(2, 2, 100, device="cuda"))
    graph.replay()
    for h in range(2):
        assert got[0][0, h].tolist() == ref.select(w[0, h].cpu().numpy(), 40, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kept, nl, nw = (torch.empty_like(x) for x in got)
    dcp.dcp_kv_evict(w, k, v, table, seq, ko, vo, new, 40, 4, kept, nl, nw, stream=s)
    s.synchronize()
    assert torch.equal(kept, got[0]) and torch.equal(nw, got[2])


def test_evict_very_long():
    """More weights than one block's shared memory holds."""
    check_evict([150000, 70001], 1, 8, 128, 600, 100, seed=4)


def test_evict_ties_zeros_and_specials():
    """Equal weights (lowest positions win), +0 with -0, infinities, NaN, negative and denormal
    weights, and rows of one value."""
    n = 700
    g = torch.Generator().manual_seed(1)
    w = torch.zeros(6, 2, n)
    w[0] = torch.randint(0, 4, (2, n), generator=g).float()
    w[1] = torch.where(torch.rand(2, n, generator=g) < 0.5, -0.0, 0.0)
    w[2] = torch.randn(2, n, generator=g)
    w[2, :, ::7] = float("nan")
    w[2, :, ::11] = float("inf")
    w[2, :, 1::3] = float("-inf")
    w[3] = 1.25
    w[4] = float("nan")
    w[5] = torch.randint(0, 50, (2, n), generator=g).float() * 2.0 ** -149
    for keep, recent in ((100, 0), (400, 30), (699, 1), (50, 50)):
        check_evict([n] * 6, 2, 16, 16, keep, recent, weights=w)


def test_evict_into_the_same_pool_and_shards():
    check_evict([90, 200, 30], 2, 64, 16, 48, 8, same_pool=True)
    seq = [100, 300, 50]
    check_evict([ref.local_len(x, 2, 4, 8) for x in seq], 2, 64, 16, 20, 3, seq=seq, shard=2, num_shards=4,
                interleave=8)


def test_evict_bad_pages_and_short_weights():
    check_evict([100, 80], 2, 64, 16, 40, 4, bad_src=((0, 1), (1, 0)), bad_dst=((0, 2), (1, 1)))
    check_evict([100, 80], 2, 64, 16, 40, 4, cap=60, new_cap=45)
    check_evict([100], 2, 64, 16, 40, 4, seq=[-3] and [100], new_cap=40)


def test_evict_many_rows():
    g = torch.Generator().manual_seed(8)
    check_evict(torch.randint(0, 60, (220,), generator=g).tolist(), 4, 16, 16, 20, 2)


def test_evict_helper_and_refusals():
    case = ref.PagedCase([50, 10], 2, 64, 16, "bf16", seed=2)
    k, v, table = case.gpu()
    w = torch.rand(2, 2, 50, device="cuda")
    k = torch.cat([k, torch.zeros_like(k)])
    v = torch.cat([v, torch.zeros_like(v)])
    new = (torch.arange(4, dtype=torch.int32, device="cuda") + case.pages).reshape(2, 2)
    kept, nl, nw = dcp.kv_evict(w, k, v, table, i32([50, 10]), new, 20, 4)
    assert nl.tolist() == [20, 10] and nw.shape == w.shape and kept.shape == (2, 2, 20)
    assert (kept[1, :, 10:] == -1).all() and (nw[1, :, 10:] == 0).all()
    with pytest.raises(dcp.DCPError):
        dcp.kv_evict(w, k, v, table, i32([50, 10]), new, 33)       # 2 pages of 16 hold 32
    with pytest.raises(dcp.DCPError):
        dcp.kv_evict(w, k, v, table, i32([50, 10]), new, 20, 21)
    with pytest.raises(ValueError):
        dcp.kv_evict(w, k, v, table, i32([50, 10]), new, 20, 4, k_out=k)
    with pytest.raises(ValueError):
        dcp.kv_evict(w[:1], k, v, table, i32([50, 10]), new, 20)


def test_refused_arguments_of_all_calls():
    """Integers that do not fit 32 bits are not cut, and outputs whose rows overlap are refused."""
    case = ref.PagedCase([50, 10], 2, 64, 16, "bf16", seed=3)
    k, v, table = case.gpu()
    seq, starts = i32([50, 10]), i32([0, 1, 2])
    q, new = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), k[0, :2].clone()
    logits, lse = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 4, device="cuda")
    w = torch.zeros(2, 2, 64, device="cuda")
    out = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    new_table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(2, 2)

    def calls(**kw):
        yield lambda: dcp.paged_attention(q, k, v, table, seq, **kw)
        yield lambda: dcp.paged_attention_pack(q, k, v, table, seq, 2, **kw)
        yield lambda: dcp.dcp_kv_append(new, new, k, v, table, seq, starts, **kw)
        yield lambda: dcp.dcp_kv_weights(logits, lse, seq, w, **kw)
        yield lambda: dcp.kv_evict(w, k, v, table, seq, new_table, 20, 4, k_out=out, v_out=out.clone(), **kw)

    for kw in (dict(interleave=(1 << 32) + 1), dict(num_shards=(1 << 32) + 1), dict(shard=1 << 32)):
        for call in calls(**kw):
            with pytest.raises(ValueError, match="32-bit"):
                call()
    for call in calls():
        call()
    with pytest.raises(dcp.DCPError, match="overlap"):
        dcp.paged_attention(q, k, v, table, seq, logits=logits[:, :1].expand(2, 4, 64))
    with pytest.raises(dcp.DCPError, match="overlap"):
        dcp.dcp_kv_weights(logits, lse, seq, w[:1].expand(2, 2, 64))
    with pytest.raises(dcp.DCPError, match="overlap"):
        dcp.dcp_kv_append(new, new, k[:, :, :1].expand_as(k), v, table, seq, starts)
    with pytest.raises(dcp.DCPError, match="overlap"):
        dcp.kv_evict(w, k, v, table, seq, new_table, 20, 4, k_out=out[:1].expand_as(out), v_out=out)


# ---- all of it together -----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,layout", [("bf16", "slots"), ("fp32", "heads")])
def test_decode_loop_of_three_ranks(dtype, layout):
    """Prompts are appended, tokens decoded, weights accumulated and the cache evicted on 3 ranks
    (emulated in turn), the partial results exchanged and combined by the library; every step's
    output is compared with attention in 64 bits over what the caches hold."""
    N, s, heads, H, D, page, R = 3, 4, 2, 6, 64, 8, 4
    dt = ref.DTYPES[dtype]
    g = torch.Generator().manual_seed(21)
    prompts = [1, 30, 77, 12]
    ranks = []
    for r in range(N):
        shape = (120, page, heads, D) if layout == "slots" else (120, heads, page, D)
        k, v = torch.full(shape, float("nan"), dtype=dt, device="cuda"), torch.full(shape, float("nan"), dtype=dt,
                                                                                  device="cuda")
        if layout != "slots":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        ranks.append(dict(k=k, v=v, table=torch.arange(R * 10, dtype=torch.int32, device="cuda").reshape(R, 10),
                          w=torch.zeros(R, heads, 80, device="cuda"), logits=torch.zeros(R, H, 80, device="cuda"),
                          mine=[[[] for _ in range(heads)] for _ in range(R)],   # (position, weight) held, per head
                          lens=None))
    tokens = [(torch.randn(n, heads, D, generator=g).to(dt), torch.randn(n, heads, D, generator=g).to(dt))
              for n in prompts]
    dense = [list(zip(a, b)) for a, b in tokens]   # request -> [(key [heads, D], value)] by position
    lens = list(prompts)
    starts = [0]
    for n in prompts:
        starts.append(starts[-1] + n)
    k_new, v_new = torch.cat([a for a, _ in tokens]).cuda(), torch.cat([b for _, b in tokens]).cuda()

    def append(new_k, new_v, starts, per_request):
        for r, c in enumerate(ranks):
            if c["lens"] is None:  # lengths over all shards
                dcp.dcp_kv_append(new_k, new_v, c["k"], c["v"], c["table"], i32(lens), i32(starts), shard=r,
                                  num_shards=N, interleave=s)
            else:  # after an eviction: the rank's own lengths, and only its own tokens
                own = [((lens[b] - 1) // s) % N == r for b in range(R)]
                c["lens"] = [x + o for x, o in zip(c["lens"], own)]
                pick = [b for b in range(R) if own[b]]
                at = np.concatenate([[0], np.cumsum(own)]).tolist()
                dcp.dcp_kv_append(new_k[pick], new_v[pick], c["k"], c["v"], c["table"], i32(c["lens"]), i32(at))
            for b in range(R):
                for p in range(lens[b] - per_request[b], lens[b]):
                    if (p // s) % N == r:
                        for h in range(heads):
                            c["mine"][b][h].append((p, 0.0))

    append(k_new, v_new, starts, prompts)
    for step in range(8):
        q = torch.randn(R, H, D, generator=g).mul_(2.0).to(dt)
        new = torch.randn(2, R, heads, D, generator=g).to(dt)
        for b in range(R):
            dense[b].append((new[0, b], new[1, b]))
            lens[b] += 1
        append(new[0].cuda(), new[1].cuda(), list(range(R + 1)), [1] * R)
        sends = []
        for r, c in enumerate(ranks):
            shards = dict(shard=r, num_shards=N, interleave=s) if c["lens"] is None else {}
            seq = i32(lens if c["lens"] is None else c["lens"])
            sends.append(dcp.paged_attention_pack(q.cuda(), c["k"], c["v"], c["table"], seq, N, logits=c["logits"],
                                                  **shards))
        out, lse = [], []
        for r in range(N):  # the exchange: rank r receives chunk r of every rank
            o, l = dcp.unpack_combine(torch.stack([x[r] for x in sends]), return_lse=True)
            out.append(o)
            lse.append(l)
        out, lse = torch.cat(out, 1), torch.cat(lse, 1)
        G = H // heads
        want, want_lse = np.zeros((R, H, D)), np.zeros((R, H))
        for b in range(R):
            for h in range(H):
                held = sorted(p for c in ranks for p, _ in c["mine"][b][h // G])
                kk = torch.stack([dense[b][p][0][h // G] for p in held])[:, None]
                vv = torch.stack([dense[b][p][1][h // G] for p in held])[:, None]
                o, l, lo, _, _ = ref.attention(q[b:b + 1, h:h + 1], [kk], [vv], 1 / math.sqrt(D))
                want[b, h], want_lse[b, h] = o[0, 0], l[0, 0]
                p_of = dict(zip(held, np.exp(lo[0][0] - l[0, 0])))
                for c in ranks:
                    c["mine"][b][h // G] = [(p, w + p_of[p]) for p, w in c["mine"][b][h // G]]
        # two roundings of a value below 4 (partial and merged) and fp32 arithmetic around them
        tol = (2 * 4 * ref.HALF[dtype] if dtype != "fp32" else 2e-5)
        assert np.abs(out.cpu().double().numpy() - want).max() <= tol
        assert np.abs(lse.cpu().double().numpy() - want_lse).max() <= 1e-4
        for r, c in enumerate(ranks):
            shards = dict(shard=r, num_shards=N, interleave=s) if c["lens"] is None else {}
            seq = i32(lens if c["lens"] is None else c["lens"])
            dcp.dcp_kv_weights(c["logits"], lse, seq, c["w"], **shards)
            for b in range(R):
                for h in range(heads):
                    w = np.array([x for _, x in c["mine"][b][h]])
                    assert np.abs(c["w"][b, h, :len(w)].cpu().double().numpy() - w).max(initial=0) <= 1e-3
        if step in (3, 6):
            keep, recent = 10, 2
            for r, c in enumerate(ranks):
                shards = dict(shard=r, num_shards=N, interleave=s) if c["lens"] is None else {}
                seq = i32(lens if c["lens"] is None else c["lens"])
                fresh = torch.arange(R * 10, dtype=torch.int32, device="cuda").reshape(R, 10) + (40 if step == 3 else 80)
                kept, nl, c["w"] = dcp.kv_evict(c["w"], c["k"], c["v"], c["table"], seq, fresh, keep, recent, **shards)
                c["table"], c["lens"] = fresh, nl.tolist()
                for b in range(R):
                    for h in range(heads):
                        sel = kept[b, h, :c["lens"][b]].tolist()
                        mine = c["mine"][b][h]
                        assert sel == sorted(sel) and len(sel) == min(len(mine), keep)
                        if len(mine) > keep:  # the kept ones weigh at least what is left out, to rounding
                            out_w = [w for i, (_, w) in enumerate(mine[:-recent]) if i not in set(sel)]
                            assert min(mine[i][1] for i in sel[:-recent]) >= max(out_w) - 2e-3
                        c["mine"][b][h] = [mine[i] for i in sel]

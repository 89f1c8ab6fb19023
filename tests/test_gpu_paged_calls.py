"""Calls of the paged cache that the documentation allows and that lie off the usual path: the same slot
named twice, lengths that name nothing, arrays wider than their content."""
from __future__ import annotations

import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref
from decode_context_attention_dcp_b200 import paged
from test_gpu_paged_cache import check_evict

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R", [2, 500])
def test_tokens_appended_to_the_same_slot(dtype, R):
    """Requests in pairs that share their page: every element of the slot is one of the two tokens', nothing else
    is written, and requests of their own pages get their token whole."""
    page, heads, D = 4, 3, 64
    k = torch.full((R, page, heads, D), -1.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, -2.0)
    # values below 256, so that bf16 tells tokens of a pair apart
    token = torch.arange(R, device="cuda") % 100 + 1
    k_new = token.to(dtype)[:, None, None].expand(R, heads, D).contiguous()
    v_new = (token + 100).to(dtype)[:, None, None].expand(R, heads, D).contiguous()
    own = torch.arange(R, device="cuda") % 10 >= 8  # the last pair of ten keep their own pages
    table = torch.where(own, torch.arange(R, device="cuda"), torch.arange(R, device="cuda") // 2 * 2)
    dcp.dcp_kv_append(k_new, v_new, k, v, table.to(torch.int32)[:, None], i32([2] * R), i32(list(range(R + 1))))
    for pool, new, fill in ((k, k_new, -1.0), (v, v_new, -2.0)):
        assert (pool[:, [0, 2, 3]] == fill).all()
        slot = pool[:, 1]
        first = torch.arange(R, device="cuda") // 2 * 2
        shared, partner = ~own & (first == torch.arange(R, device="cuda")), (first + 1).clamp(max=R - 1)
        assert torch.equal(slot[own], new[own])
        either = (slot == new) | (slot == new[partner])
        assert either[shared].all()
        assert (slot[~own & ~shared] == fill).all()


def test_the_same_results_without_the_compiled_binding(monkeypatch):
    """Every call made by the Python code instead of the binding."""
    k = torch.randn(12, 16, 2, 64, device="cuda").to(torch.bfloat16)
    v, q = torch.randn_like(k), torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    table, seq, starts = i32([[0, 1, 2], [3, 4, 5]]), i32([40, 17]), i32([0, 1, 2])
    new = torch.randn(2, 2, 64, device="cuda").to(torch.bfloat16)

    def step():
        kk, vv, w = k.clone(), v.clone(), torch.zeros(2, 2, 48, device="cuda")
        logits = torch.zeros(2, 4, 48, device="cuda")
        dcp.dcp_kv_append(new, new + 1, kk, vv, table, seq, starts)
        out, lse = dcp.paged_attention(q, kk, vv, table, seq, logits=logits)
        send = dcp.paged_attention_pack(q, kk, vv, table, seq, 2)
        dcp.dcp_kv_weights(logits, lse, seq, w)
        kept, lens, weights = dcp.kv_evict(w, kk, vv, table, seq, table + 6, 20, 4)
        return kk, vv, out, lse, send.view(torch.int16), w, kept, lens, weights

    want = step()
    monkeypatch.setattr(paged, "_native", paged._NoBinding)
    for a, b in zip(step(), want):
        assert torch.equal(a, b)


def test_eviction_refuses_integers_past_64_bits():
    k = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    w, table, new = torch.rand(1, 2, 40, device="cuda"), i32([[0, 1, 2]]), i32([[4, 5]])
    for recent in ((1 << 64) + 1, -(1 << 64) + 1):
        with pytest.raises(ValueError, match="64-bit"):
            dcp.kv_evict(w, k, k.clone(), table, i32([40]), new, 20, recent)
    for recent in (1 << 40, 21, -1):
        with pytest.raises(dcp.DCPError, match="recent"):
            dcp.kv_evict(w, k, k.clone(), table, i32([40]), new, 20, recent)


@pytest.mark.parametrize("interleave", [1, 3])
def test_tokens_that_follow_an_eviction_in_a_captured_step(interleave):
    """Ranks of lengths of their own: a step captured once, in which each rank appends the tokens it owns (lengths of
    0 leave the others out), replayed for twelve tokens."""
    N, R, heads, D, page = 2, 3, 2, 64, 4
    total = i32([7, 20, 1])
    k_new, v_new = (torch.zeros(R, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ranks = []
    for r in range(N):
        k = torch.full((18, page, heads, D), -1.0, dtype=torch.bfloat16, device="cuda")
        ranks.append(dict(k=k, v=k.clone(), lens=i32([2 + r, 5, 0]), table=torch.arange(18, dtype=torch.int32,
                                                                                       device="cuda").reshape(R, 6)))
    starts = i32(list(range(R + 1)))

    def step():
        total.add_(1)
        for r, c in enumerate(ranks):
            own = (total - 1) // interleave % N == r
            c["lens"] += own
            dcp.dcp_kv_append(k_new, v_new, c["k"], c["v"], c["table"], torch.where(own, c["lens"], 0), starts)

    held = [[[-1.0] * int(n) for n in c["lens"]] for c in ranks]  # per rank and request: the values of its slots
    first = total.tolist()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        dcp.dcp_kv_append(k_new, v_new, ranks[0]["k"], ranks[0]["v"], ranks[0]["table"], i32([0] * R), starts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(12):
        k_new.copy_((torch.arange(R) + 1 + 10 * i)[:, None, None].expand(R, heads, D))
        v_new.copy_(k_new + 1)
        graph.replay()
        for b in range(R):
            held[(first[b] + i) // interleave % N][b].append(float(b + 1 + 10 * i))
    for r, c in enumerate(ranks):
        assert c["lens"].tolist() == [len(x) for x in held[r]]
        for b in range(R):
            for pool, more in (("k", 0), ("v", 1)):
                slots = c[pool][6 * b:6 * b + 6].reshape(6 * page, heads, D).float()
                want = [x + more * (x > 0) for x in held[r][b]] + [-1.0] * (6 * page - len(held[r][b]))
                assert (slots == torch.tensor(want, device="cuda")[:, None, None]).all(), (r, b, pool)


@pytest.mark.parametrize("lens,seq", [([0, 100], [-3, 1 << 30]), ([0, 100] * 115, [-(1 << 31), (1 << 31) - 1] * 115),
                                      ([20011, 0, 20011], [20012, -1, 1 << 30]), ([0, 60000], [-5, 1 << 30])])
def test_eviction_of_negative_lengths_and_lengths_past_the_arrays(lens, seq):
    """In every selection kernel: a negative length is 0 (nothing kept, new weights all 0), a longer one is cut."""
    check_evict(lens, 2 if len(lens) < 10 else 4, 8, 16, 40, 5, seq=seq)
    check_evict(lens, 1, 8, 64, 40, 5, seq=seq, new_cap=47)


@pytest.mark.parametrize("n,keep,wide", [(n, keep, wide) for n, keep in ((100, 30), (3000, 500), (20000, 1000), (5, 40))
                                         for wide in (4097, 49153, 131072) if wide > n])
def test_eviction_in_arrays_wider_than_their_content(n, keep, wide):
    """Weights and tables with room for far more positions than are held, as a server keeps them: the same as
    in arrays of the content's size."""
    heads, page, lens = 2, 16, [n, n // 2, 0]
    case = ref.PagedCase(lens, heads, 16, page, "bf16", seed=n)
    k, v, table = case.gpu()
    w = torch.rand(3, heads, n, generator=torch.Generator().manual_seed(n)).cuda()
    new = torch.randperm(3 * (keep // page + 1), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    new = new.reshape(3, -1).cuda()
    w_wide = torch.full((3, heads, wide), float("nan"), device="cuda")  # not held: never looked at
    w_wide[:, :, :n] = w
    t_wide = torch.full((3, wide // page + 1), -1, dtype=torch.int32, device="cuda")
    t_wide[:, :table.shape[1]] = table
    t_new = torch.full((3, wide // page + 1), -1, dtype=torch.int32, device="cuda")
    t_new[:, :new.shape[1]] = new
    results = []
    for weights, src, dst in ((w, table, new), (w_wide, t_wide, t_new)):
        ko = torch.zeros(new.numel(), page, heads, 16, dtype=k.dtype, device="cuda")
        vo = torch.zeros_like(ko)
        kept, nl, nw = dcp.kv_evict(weights, k, v, src, i32(lens), dst, keep, keep // 8, k_out=ko, v_out=vo)
        results.append((kept, nl, ko, vo, nw))
    for a, b in zip(results[0][:4], results[1][:4]):
        assert torch.equal(a, b)
    assert torch.equal(results[1][4][:, :, :results[0][4].shape[2]], results[0][4])
    assert (results[1][4][:, :, results[0][4].shape[2]:] == 0).all()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 20), (256, 16)])
def test_long_fp32_sums_keep_their_precision(D, page):
    """512 requests that share 20011 positions: some 300 tiles per block, so sums of thousands of positions.

    The error's RMS relative to the result's, from the arithmetic, each part independent and of random sign: a
    logit's products with factors of two tf32 parts, the second cut to 10 bits (up to 2^-21 of a factor, RMS half
    of it over sqrt(3) each, twice): 2e-7 of a logit of standard deviation 1; its sum's roundings, about 8 of
    2^-24: 2e-7; exp2 and its argument, 2^-22 and 2^-24 times 8: 4e-7 together; weight and value in the product,
    2e-7; the fp32 sums of 360 tiles, a random walk of 2^-25: 19 times 3e-8 of a sum that itself grows as one:
    4e-7.  In all 7e-7; the bound is 2e-6.  (The same sums left to the product units: 5e-6; products of one
    tf32 part: 1e-4.)"""
    B, n = 512, 20011
    case = ref.PagedCase([n], 1, D, page, "fp32", seed=D + page)
    k, v, table = case.gpu()
    q = torch.randn(B, 2, D, generator=torch.Generator().manual_seed(D)).cuda()
    out, lse = dcp.paged_attention(q, k, v, table.expand(B, -1), i32([n] * B))
    keys, values = case.keys[0][:, 0].double().cuda(), case.values[0][:, 0].double().cuda()
    x = q.double().reshape(2 * B, D) @ keys.t() * (1 / D ** 0.5)
    want = (x.softmax(1) @ values).reshape(B, 2, D)
    assert float((out.double() - want).norm() / want.norm()) <= 2e-6
    # ln of a sum whose terms have relative errors of 1e-6 at most, rounded at its size of about 10.4
    assert float((lse.double() - x.logsumexp(1).reshape(B, 2)).abs().max()) <= 1e-6 + 4 * 2.0 ** -21

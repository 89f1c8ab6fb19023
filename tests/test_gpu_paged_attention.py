"""Attention of one new token over a paged cache against the definition in 64 bits, element by
element, within bounds that follow from the arithmetic (paged_ref.assert_attention).  Everything
in the pool that a request does not hold is NaN, table entries past a length name no page, and
outputs carry guard bands."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu


def query(B, H, D, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed + 77)
    return torch.randn(B, H, D, generator=g).mul_(std).to(ref.DTYPES[dtype])


def check(case: ref.PagedCase, H: int, std=1.0, base_e=True, scale=None, held=None, lens=None, with_logits=True, **kw):
    """Runs the plain and (H even) the packed form of one case and compares both."""
    B, D, dtype = len(case.lens), case.D, case.dtype
    q = query(B, H, D, dtype, case.seed, std)
    k, v, table = case.gpu()
    seq = torch.tensor(case.lens if lens is None else lens, dtype=torch.int32, device="cuda")
    scale_ref = float(np.float32(1 / math.sqrt(D) if scale is None else scale))
    r = ref.attention(q, case.keys, case.values, scale_ref, held)
    n_max = max((x.shape[0] for x in case.keys), default=0)
    out, lse = Guarded((B, H, D), q.dtype), Guarded((B, H), torch.float32)
    cap = max(1, n_max - 3)
    logits = Guarded((B, H, cap), torch.float32) if with_logits else None
    if logits is not None:
        logits.tensor.fill_(7.5)
    dq = q.cuda()
    dcp.dcp_paged_attention(dq, k, v, table, seq, out.tensor, lse.tensor, scale=scale, is_lse_base_on_e=base_e,
                            logits=logits.tensor if logits is not None else None, **kw)
    out.check(), lse.check()
    what = f"{dtype} {case.layout} B{B} H{H}/{case.heads} D{D} page{case.page} n{n_max}"
    ref.assert_attention(out.tensor, lse.tensor, r, n_max, dtype, base_e, what)
    if logits is not None:
        logits.check()
        got = logits.tensor.cpu().double().numpy()
        for b in range(B):
            n = min(cap, case.keys[b].shape[0])
            want, bound = r[2][b][:, :n], ref.logit_bound(r[4][b][:, :n], D, dtype)
            fin = np.isfinite(want)
            assert np.array_equal(got[b, :, :n][~fin], want[~fin]), what
            assert (np.abs(got[b, :, :n][fin] - want[fin]) <= bound[fin]).all(), f"{what}: logits"
            assert (got[b, :, n:] == 7.5).all(), f"{what}: logits written past the held positions"
    if H % 2 == 0:
        P = dcp.dcp_lse_pack_dim(q.dtype)
        send = Guarded((2, B, H // 2, D + P), q.dtype)
        dcp.dcp_paged_attention_pack(dq, k, v, table, seq, send.tensor, 2, scale=scale, is_lse_base_on_e=base_e, **kw)
        send.check()
        # the same bits as the plain form, packed
        want = dcp.pack(out.tensor, lse.tensor, 2)
        assert torch.equal(send.tensor.view(torch.uint8), want.view(torch.uint8)), f"{what}: packed form differs"
    return out.tensor, lse.tensor


RAGGED = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200]


# A table of a few tiles gives each request a cluster of blocks; one that could hold more has the
# tiles shared evenly over the device: the tests below run both on the same requests.
WIDE = 700


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [8, 16, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("width", [None, WIDE])
def test_head_dims_and_lengths(dtype, D, width):
    check(ref.PagedCase(RAGGED, 2, D, 16, dtype, seed=D, width=width), H=8)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[1], [64], [65, 0], [300], [129, 500, 17], [1000, 2, 0, 600], [1500]])
def test_few_requests(dtype, D, lens):
    """Clusters of one to eight blocks, some of them without a tile."""
    check(ref.PagedCase(lens, 2, D, 16, dtype, seed=len(lens) + D), H=6)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,heads", [(1, 1), (3, 3), (5, 1), (8, 8), (14, 2), (16, 1), (17, 1), (32, 1), (33, 1),
                                     (64, 2), (100, 2), (128, 1), (96, 8)])
@pytest.mark.parametrize("width", [None, WIDE])
def test_head_groups(dtype, H, heads, width):
    check(ref.PagedCase([0, 1, 37, 150, 64], heads, 64, 16, dtype, seed=H, width=width), H=H)


@pytest.mark.parametrize("H,heads,D", [(48, 1, 128), (33, 1, 256), (40, 2, 192), (16, 1, 256), (20, 1, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("width", [None, WIDE])
def test_wide_groups_of_wide_heads(dtype, H, heads, D, width):
    check(ref.PagedCase([70, 0, 129], heads, D, 32, dtype, seed=H + D, width=width), H=H)


@pytest.mark.parametrize("page", [1, 2, 5, 8, 13, 16, 24, 32, 48, 64, 100, 128, 256])
@pytest.mark.parametrize("layout", ["slots", "heads", "mixed"])
@pytest.mark.parametrize("width", [None, 12000])
def test_pages_and_layouts(page, layout, width):
    check(ref.PagedCase(RAGGED, 2, 128, page, "bf16", layout, seed=page, width=width), H=8)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("layout", ["heads", "mixed"])
def test_layouts_of_other_types(dtype, layout):
    check(ref.PagedCase(RAGGED, 3, 96, 24, dtype, layout, seed=5), H=6)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("base_e", [True, False])
def test_peaked_logits_and_bases(dtype, base_e):
    """Logits of standard deviation 6 over 1500 positions, both LSE bases."""
    check(ref.PagedCase([1500, 3, 700], 2, 64, 16, dtype, seed=9), H=4, std=6.0, base_e=base_e)


@pytest.mark.parametrize("scale", [0.0, -0.5, 1.0])
def test_scales(scale):
    check(ref.PagedCase([100, 1], 1, 64, 16, "bf16", seed=4), H=4, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_long_request_is_split(dtype):
    """One long request beside short ones: its length is divided over the whole device."""
    check(ref.PagedCase([5001, 1, 0, 33], 1, 128, 16, dtype, seed=2), H=8)
    check(ref.PagedCase([9000], 1, 64, 64, dtype, seed=3), H=2)


@pytest.mark.parametrize("B", [1, 2, 150, 257, 700])
def test_batches(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 90, (B,), generator=g).tolist()
    check(ref.PagedCase(lens, 2, 64, 16, "bf16", seed=B), H=4)


def test_empty_batch_and_empty_cache():
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = dcp.paged_attention(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), k, k,
                                   torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                                   torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # a table without columns, and a pool without pages: nothing is held
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    seq = torch.tensor([5, 0, -3], dtype=torch.int32, device="cuda")
    for kk, table in ((k, torch.zeros(3, 0, dtype=torch.int32, device="cuda")),
                      (k[:0], torch.zeros(3, 2, dtype=torch.int32, device="cuda"))):
        out, lse = dcp.paged_attention(q, kk, kk, table, seq)
        assert (out == 0).all() and (lse == float("-inf")).all()


def test_lengths_past_the_table_and_negative_are_cut():
    case = ref.PagedCase([64, 48, 0], 2, 64, 16, "bf16", width=4, seed=6)
    check(case, H=4, lens=[1 << 30, 48, -7])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page", [8, 16, 20])
def test_pages_outside_the_pool_are_not_held(dtype, page):
    """Entries -1, num_pages and far values inside a length: their positions do not count, and
    their logits are -inf."""
    case = ref.PagedCase([100, 90, 40, 17], 2, 64, page, dtype, seed=8)
    held = []
    for b, n in enumerate(case.lens):
        bad = {0: [1], 1: [0, 2], 2: list(range(5)), 3: []}[b]
        for j in bad:
            if j < case.width:
                case.table[b, j] = [-1, case.pages, 2 ** 31 - 1, -2 ** 31][(b + j) % 4]
        held.append([p for p in range(n) if p // page not in bad])
    check(case, H=4, held=held)


@pytest.mark.parametrize("n,s", [(2, 1), (4, 16), (3, 5), (8, 64), (64, 1 << 30), (64, 2 ** 31 - 1)])
def test_shards(n, s):
    """seq_lens over all shards: each rank attends to its own local length."""
    seq = [0, 1, 2, 15, 16, 17, 63, 64, 100, 300, 301]
    for shard in sorted({0, 1, n - 1}):
        if s < 1000:
            local = [ref.local_len(x, shard, n, s) for x in seq]
        else:
            local = seq if shard == 0 else [0] * len(seq)
        check(ref.PagedCase(local, 2, 64, 16, "bf16", seed=shard), H=4, lens=seq, shard=shard, num_shards=n,
              interleave=s, with_logits=False)


def test_strided_query_and_table_and_logits():
    case = ref.PagedCase([33, 70], 2, 64, 16, "bf16", seed=11)
    k, v, table = case.gpu()
    wide = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + case.width] = table
    q = query(2, 4, 64, "bf16", 11)
    qkv = torch.randn(2, 4, 3, 64, device="cuda").to(torch.bfloat16)
    qkv[:, :, 1] = q.cuda()
    big = torch.full((2, 8, 100), 3.0, device="cuda")
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    out, lse = dcp.paged_attention(qkv[:, :, 1], k, v, wide[:, 2:2 + case.width], seq, logits=big[:, 1::2, 5:])
    r = ref.attention(q, case.keys, case.values, float(np.float32(0.125)))
    ref.assert_attention(out, lse, r, 70, "bf16")
    want, l2 = dcp.paged_attention(q.cuda(), k, v, table, seq)
    assert torch.equal(out, want) and torch.equal(lse, l2)
    got = big.cpu()
    assert (got[:, 0::2] == 3).all() and (got[:, :, :5] == 3).all()
    for b, n in enumerate(case.lens):
        bound = ref.logit_bound(r[4][b], 64, "bf16")
        assert (np.abs(got[b, 1::2, 5:5 + n].double().numpy() - r[2][b]) <= bound).all()
        assert (got[b, 1::2, 5 + n:] == 3).all()


def test_broadcast_query_and_shared_pages():
    """Requests that share pages (a common prefix) and one query row for all heads (stride 0)."""
    case = ref.PagedCase([64], 1, 64, 16, "bf16", seed=12)
    k, v, table = case.gpu()
    q = query(1, 1, 64, "bf16", 12).cuda()
    lens = [64, 10, 64, 33]
    out, lse = dcp.paged_attention(q.expand(4, 6, 64), k, v, table.expand(4, case.width),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"))
    r = ref.attention(q.cpu().expand(4, 6, 64), [case.keys[0][:n] for n in lens], [case.values[0][:n] for n in lens],
                      float(np.float32(0.125)))
    ref.assert_attention(out, lse, r, 64, "bf16")


def test_pool_past_32_bit_offsets():
    """A key pool of more than 2^31 elements whose last pages are used."""
    P, page, D = (1 << 31) // (16 * 128) + 10, 16, 128
    case = ref.PagedCase([50, 3], 1, D, page, "bf16", seed=13)
    k = torch.empty(P, page, 1, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(P, page, 1, D, dtype=torch.bfloat16, device="cuda")
    k[P - case.pages:], v[P - case.pages:] = case.k.cuda(), case.v.cuda()
    table = case.table.clone()
    table[table < 2 ** 30] += P - case.pages
    q = query(2, 4, D, "bf16", 13)
    out, lse = dcp.paged_attention(q.cuda(), k, v, table.cuda(), torch.tensor(case.lens, dtype=torch.int32,
                                                                              device="cuda"))
    r = ref.attention(q, case.keys, case.values, float(np.float32(1 / math.sqrt(D))))
    ref.assert_attention(out, lse, r, 50, "bf16")


def test_special_values():
    """Keys of -inf logits add nothing; a row of -inf logits only is empty; NaN and +inf logits
    give NaN, as the formula does; other rows stay as they are."""
    case = ref.PagedCase([40, 40, 40, 40], 1, 64, 16, "bf16", seed=14)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    q[:, 1, 1] = 1.0
    k, v, table = case.gpu()
    inf = float("inf")

    def key(b, p):
        return k[int(case.table[b, p // 16]), p % 16, 0]

    for p in range(40):
        if p % 3:
            key(0, p)[0] = -inf
        key(1, p)[0] = -inf
    key(2, 5)[0] = inf
    key(3, 39)[0] = float("nan")
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    out, lse = dcp.paged_attention(q.cuda(), k, v, table, seq)
    held = [[p for p in range(40) if p % 3 == 0], [], range(40), range(40)]
    for kk in case.keys[:2]:
        kk[torch.isinf(kk)] = 0
    r = ref.attention(q, case.keys, case.values, float(np.float32(0.125)), held)
    ref.assert_attention(out[:2], lse[:2], tuple(x[:2] for x in r), 40, "bf16")
    assert torch.isnan(out[2:]).all()
    assert torch.isnan(lse[3]).all() and not torch.isfinite(lse[2]).any()


@pytest.mark.parametrize("lens", [[3000, 17, 900], [200, 17, 90]])
def test_same_bits_every_time(lens):
    case = ref.PagedCase(lens, 2, 128, 16, "bf16", seed=15)
    k, v, table = case.gpu()
    q = query(3, 8, 128, "bf16", 15).cuda()
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    first = dcp.paged_attention(q, k, v, table, seq)
    for _ in range(5):
        again = dcp.paged_attention(q, k, v, table, seq)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_other_stream_and_two_at_once():
    """Calls on two streams at the same time, each with its own workspace."""
    case = ref.PagedCase([2000, 5, 1200, 0], 2, 128, 16, "bf16", seed=16)
    k, v, table = case.gpu()
    q = query(4, 8, 128, "bf16", 16).cuda()
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    want = dcp.paged_attention(q, k, v, table, seq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for i in range(20):
        s = streams[i % 2]
        o, l = torch.empty_like(want[0]), torch.empty_like(want[1])
        s.wait_stream(torch.cuda.current_stream())
        dcp.dcp_paged_attention(q, k, v, table, seq, o, l, stream=s if i % 4 else s.cuda_stream)
        results.append((o, l))
    torch.cuda.synchronize()
    for o, l in results:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("width", [None, WIDE])
def test_graph_replay_with_other_lengths(width):
    """Captured once (two calls in one graph), replayed with other lengths and queries."""
    case = ref.PagedCase([900, 64, 200], 2, 64, 16, "bf16", seed=17, width=width)
    k, v, table = case.gpu()
    q = query(3, 8, 64, "bf16", 17).cuda()
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    dcp.paged_attention(q, k, v, table, seq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = dcp.paged_attention(q, k, v, table, seq)
        send = dcp.paged_attention_pack(q, k, v, table, seq, 4)
    for lens in ([900, 64, 200], [1, 0, 199], [0, 0, 0], [512, 33, 16]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(query(3, 8, 64, "bf16", 17 + lens[0]))
        graph.replay()
        r = ref.attention(q.cpu(), [x[:n] for x, n in zip(case.keys, lens)],
                          [x[:n] for x, n in zip(case.values, lens)], float(np.float32(0.125)))
        ref.assert_attention(out, lse, r, 900, "bf16", what=str(lens))
        assert torch.equal(send.view(torch.uint8), dcp.pack(out, lse, 4).view(torch.uint8))


def test_own_workspace_and_refusals():
    case = ref.PagedCase([100], 2, 64, 16, "bf16", seed=18)
    k, v, table = case.gpu()
    q = query(1, 4, 64, "bf16", 18).cuda()
    seq = torch.tensor([100], dtype=torch.int32, device="cuda")
    want, _ = dcp.paged_attention(q, k, v, table, seq)
    n = dcp.paged_attention_workspace(q, k)
    out, lse = torch.empty_like(want), torch.empty(1, 4, device="cuda")
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    dcp.dcp_paged_attention(q, k, v, table, seq, out, lse, workspace=ws)
    assert torch.equal(out, want)
    if n > 16:
        with pytest.raises(dcp.DCPError, match="workspace"):
            dcp.dcp_paged_attention(q, k, v, table, seq, out, lse, workspace=ws[:n - 16])
    with pytest.raises(ValueError, match="workspace"):
        dcp.dcp_paged_attention(q, k, v, table, seq, out, lse, workspace=ws[:1].expand(n))
    bad = [dict(q=q.float()), dict(q=q[..., ::2]), dict(table=table.long()), dict(table=table[:, :0].expand(2, 0)),
           dict(seq=seq.long()), dict(seq=seq.repeat(2)), dict(k=k[..., :32]), dict(v=v.half())]
    for kw in bad:
        a = dict(dict(q=q, k=k, v=v, table=table, seq=seq), **kw)
        with pytest.raises((ValueError, dcp.DCPError)):
            dcp.paged_attention(a["q"], a["k"], a["v"], a["table"], a["seq"])
    with pytest.raises(ValueError):
        dcp.paged_attention(q, k, v, table, seq, logits=torch.zeros(1, 4, 8, dtype=torch.float16, device="cuda"))
    with pytest.raises(dcp.DCPError):
        dcp.paged_attention(q, k, v, table, seq, scale=math.nan)
    with pytest.raises(dcp.DCPError):
        dcp.paged_attention(q, k, v, table, seq, shard=2, num_shards=2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page", [16, 5])
def test_broadcast_cache_and_shared_tensor(dtype, page):
    """One key head seen as four (stride 0) and values that are the keys."""
    case = ref.PagedCase([50, 17], 1, 64, page, dtype, seed=31)
    k, _, table = case.gpu()
    q = query(2, 8, 64, dtype, 31)
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    out, lse = dcp.paged_attention(q.cuda(), k.expand(-1, -1, 4, -1), k.expand(-1, -1, 4, -1), table, seq)
    keys = [x.expand(-1, 4, -1) for x in case.keys]
    r = ref.attention(q, keys, keys, float(np.float32(0.125)))
    ref.assert_attention(out, lse, r, 50, dtype)


@pytest.mark.parametrize("page", [16, 24, 5])
def test_a_page_named_twice_and_wide_tables(page):
    """A table that names one page several times, with room for many more than are used."""
    case = ref.PagedCase([2 * page, page], 2, 64, page, "bf16", seed=32)
    k, v, table = case.gpu()
    wide = torch.full((2, 4000), -1, dtype=torch.int32, device="cuda")
    wide[0, :5] = table[0, 0]
    wide[1, 0], wide[1, 1], wide[1, 2] = table[0, 1], table[1, 0], table[0, 1]
    lens = [5 * page - 3, 2 * page + 1]
    q = query(2, 6, 64, "bf16", 32)
    out, lse = dcp.paged_attention(q.cuda(), k, v, wide, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    first, second = slice(0, page), slice(page, 2 * page)
    keys, values = [], []
    for src, dst in ((case.keys, keys), (case.values, values)):
        dst.append(torch.cat([src[0][first]] * 5)[:lens[0]])
        dst.append(torch.cat([src[0][second], src[1][first], src[0][second]])[:lens[1]])
    r = ref.attention(q, keys, values, float(np.float32(0.125)))
    ref.assert_attention(out, lse, r, max(lens), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_forty_thousand_positions(dtype):
    check(ref.PagedCase([40003], 1, 64, 32, dtype, seed=33), H=2, with_logits=False)


def test_integer_scale_and_keyword_streams():
    case = ref.PagedCase([30], 1, 64, 16, "bf16", seed=34)
    k, v, table = case.gpu()
    q = query(1, 2, 64, "bf16", 34, std=0.1).cuda()
    seq = torch.tensor([30], dtype=torch.int32, device="cuda")
    one, two = dcp.paged_attention(q, k, v, table, seq, scale=1), dcp.paged_attention(q, k, v, table, seq, scale=1.0)
    assert torch.equal(one[0], two[0])
    out, lse = torch.empty_like(q), torch.empty(1, 2, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dcp.dcp_paged_attention(q, k, v, table, seq, out, lse, scale=1.0, stream=s)
    s.synchronize()
    assert torch.equal(out, two[0]) and torch.equal(lse, two[1])


def test_capture_without_a_call_before():
    """A graph captured by a process that has not launched any of these kernels."""
    code = """
import torch, decode_context_attention_dcp_b200 as dcp
dcp.library()
k = torch.randn(8, 16, 2, 64, device="cuda").bfloat16(); v = torch.randn_like(k)
q = torch.randn(2, 4, 64, device="cuda").bfloat16()
t = torch.arange(8, dtype=torch.int32, device="cuda").reshape(2, 4)
n = torch.tensor([50, 3], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = dcp.paged_attention(q, k, v, t, n)
g.replay()
torch.cuda.synchronize()
want = dcp.paged_attention(q, k, v, t, n)
assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert res.returncode == 0 and "captured" in res.stdout, res.stderr[-2000:]


def test_no_wait_ran_out():
    """Last: every copy of the tests above arrived in time."""
    assert dcp.dcp_wait_timeouts() == 0

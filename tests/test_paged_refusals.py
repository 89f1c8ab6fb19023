"""The paged-cache calls without a GPU: the host-side checks of the C ABI and of the binding, and
the reference's own consistency.  Validation runs before any CUDA call, so fake (never
dereferenced) device addresses do."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref
from decode_context_attention_dcp_b200.paged import _PagedKV

OK, INVALID, DTYPE, MISALIGNED, SHAPE = 0, 1, 2, 3, 4
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return dcp.library()


def cache(**kw) -> _PagedKV:
    a = dict(k=A, v=A, block_table=A, num_pages=10, k_stride_page=16 * 2 * 128, k_stride_slot=2 * 128,
             k_stride_head=128, v_stride_page=16 * 2 * 128, v_stride_slot=2 * 128, v_stride_head=128, table_stride=4,
             max_pages=4, page_size=16, heads=2, head_dim=128, dtype=0)
    a.update(kw)
    return _PagedKV(**a)


def attend(lib, kv=None, pack=None, **kw):
    a = dict(q=A, seq=A, out=A, lse=A, logits=None, B=3, H=8, qb=8 * 128, qh=128, lb=0, lh=0, cap=0, scale=0.1,
             shard=0, n=1, inter=1, base=1, ws=A, wsb=1 << 40)
    a.update({k: v for k, v in kw.items() if k in a})
    kv = kv if kv is not None else cache(**{k: v for k, v in kw.items() if k not in a})
    tail = (a["qb"], a["qh"], a["lb"], a["lh"], a["cap"], a["scale"], a["shard"], a["n"], a["inter"], a["base"],
            a["ws"], a["wsb"], None)
    if pack is None:
        return lib.dcp_paged_attention(kv, a["q"], a["seq"], a["out"], a["lse"], a["logits"], a["B"], a["H"], *tail)
    return lib.dcp_paged_attention_pack(kv, a["q"], a["seq"], a["out"], a["logits"], a["B"], a["H"], pack, *tail)


def append(lib, **kw):
    a = dict(kn=A, vn=A, seq=A, qsl=A, T=5, R=2, kt=256, kh=128, vt=256, vh=128, shard=0, n=1, inter=1)
    a.update({k: v for k, v in kw.items() if k in a})
    kv = cache(**{k: v for k, v in kw.items() if k not in a})
    return lib.dcp_kv_append(kv, a["kn"], a["vn"], a["seq"], a["qsl"], a["T"], a["R"], a["kt"], a["kh"], a["vt"],
                             a["vh"], a["shard"], a["n"], a["inter"], None)


def evict(lib, dst=None, **kw):
    a = dict(seq=A, w=A, nw=A, kept=A, nl=A, B=3, cap=64, ncap=32, wb=128, wh=64, nb=64, nh=32, keep=32, recent=4,
             shard=0, n=1, inter=1)
    a.update({k: v for k, v in kw.items() if k in a})
    src = cache(**{k: v for k, v in kw.items() if k not in a})
    return lib.dcp_kv_evict(src, dst if dst is not None else cache(), a["seq"], a["w"], a["nw"], a["kept"], a["nl"],
                            a["B"], a["cap"], a["ncap"], a["wb"], a["wh"], a["nb"], a["nh"], a["keep"], a["recent"],
                            a["shard"], a["n"], a["inter"], None)


def weigh(lib, **kw):
    a = dict(lo=A, lse=A, seq=A, w=A, B=3, H=8, heads=2, cap=64, lb=512, lh=64, sb=8, sh=1, wb=128, wh=64, shard=0,
             n=1, inter=1, base=1)
    a.update(kw)
    return lib.dcp_kv_weights(*a.values(), None)


CALLS = [attend, lambda lib, **kw: attend(lib, pack=4, **kw), append, evict]


@pytest.mark.parametrize("call", CALLS, ids=["attention", "attention_pack", "append", "evict"])
def test_cache_rejections(lib, call):
    zero = {"T": 0} if call is append else {"B": 0}
    for bad in (dict(dtype=3), dict(dtype=-1)):
        assert call(lib, **bad) == DTYPE
    for bad in (dict(head_dim=0), dict(head_dim=264), dict(heads=0), dict(page_size=0), dict(num_pages=-1),
                dict(max_pages=-1), dict(max_pages=1 << 31), dict(max_pages=1 << 27), dict(k_stride_page=-8),
                dict(v_stride_slot=-128), dict(table_stride=-1), dict(k=None), dict(v=None), dict(block_table=None),
                dict(shard=-1), dict(shard=1), dict(n=0), dict(n=65), dict(inter=0), dict(seq=None)):
        assert call(lib, **bad) == INVALID, bad
        assert "dcp_" in dcp.dcp_last_error()
    for bad in (dict(head_dim=100), dict(k=A + 8), dict(v=A + 2), dict(block_table=A + 2), dict(k_stride_slot=260),
                dict(v_stride_head=129), dict(head_dim=6, dtype=2), dict(seq=A + 1)):
        assert call(lib, **bad) == MISALIGNED, bad
    assert call(lib, **zero) == OK
    assert dcp.dcp_last_error() == ""


def test_null_cache(lib):
    null = ctypes.POINTER(_PagedKV)()
    assert attend(lib, kv=null) == INVALID
    assert evict(lib, dst=null) == INVALID


@pytest.mark.parametrize("pack", [None, 4])
def test_attention_rejections(lib, pack):
    for bad in (dict(B=-1), dict(H=0), dict(B=1 << 30), dict(qb=-8), dict(logits=A, lb=-1), dict(logits=A, cap=-1),
                dict(logits=A, cap=1 << 31), dict(scale=math.nan), dict(scale=math.inf), dict(q=None),
                dict(out=None)):
        assert attend(lib, pack=pack, **bad) == INVALID, bad
    for bad in (dict(q=A + 8), dict(out=A + 4), dict(logits=A + 2, cap=8), dict(qh=132)):
        assert attend(lib, pack=pack, **bad) == MISALIGNED, bad
    assert attend(lib, pack=pack, H=9) == SHAPE
    assert attend(lib, lse=None) == INVALID
    assert attend(lib, lse=A + 2) == MISALIGNED
    assert attend(lib, pack=3) == SHAPE
    assert attend(lib, pack=0) == INVALID
    assert attend(lib, pack=65) == INVALID


def test_workspace_rejections(lib):
    assert lib.dcp_paged_attention_workspace(9, 2, 128, 0) == -1
    assert lib.dcp_paged_attention_workspace(8, 0, 128, 0) == -1
    assert lib.dcp_paged_attention_workspace(8, 2, 512, 0) == -1
    assert lib.dcp_paged_attention_workspace(8, 2, 128, 9) == -1
    assert lib.dcp_paged_attention_workspace(8, 2, 128, 0) >= 0


def test_append_rejections(lib):
    for bad in (dict(T=-1), dict(R=-1), dict(T=1 << 31), dict(T=1 << 30), dict(kt=-256), dict(vh=-8), dict(kn=None),
                dict(vn=None), dict(qsl=None)):
        assert append(lib, **bad) == INVALID, bad
    for bad in (dict(kn=A + 8), dict(vn=A + 4), dict(kt=250), dict(vh=100), dict(qsl=A + 2)):
        assert append(lib, **bad) == MISALIGNED, bad
    assert append(lib, R=0) == OK


def test_weights_rejections(lib):
    for bad in (dict(B=-1), dict(H=0), dict(heads=0), dict(B=1 << 30), dict(cap=-1), dict(cap=1 << 31), dict(lb=-1),
                dict(wh=-1), dict(lo=None), dict(lse=None), dict(seq=None), dict(w=None), dict(n=0), dict(shard=2),
                dict(inter=0)):
        assert weigh(lib, **bad) == INVALID, bad
    assert weigh(lib, H=7) == SHAPE
    for bad in (dict(lo=A + 2), dict(lse=A + 1), dict(w=A + 2), dict(seq=A + 3)):
        assert weigh(lib, **bad) == MISALIGNED, bad
    assert weigh(lib, B=0) == OK
    assert weigh(lib, cap=0) == OK


def test_evict_rejections(lib):
    for bad in (dict(B=-1), dict(B=1 << 30), dict(keep=0), dict(keep=1 << 31), dict(recent=-1), dict(recent=33),
                dict(cap=-1), dict(ncap=31), dict(keep=65, ncap=65), dict(wb=-1), dict(nh=-1), dict(w=None),
                dict(nw=None), dict(kept=None), dict(nl=None)):
        assert evict(lib, **bad) == INVALID, bad
    for other in (dict(heads=4), dict(head_dim=64), dict(dtype=1)):
        assert evict(lib, dst=cache(**other)) == INVALID, other
    for bad in (dict(w=A + 2), dict(nw=A + 1), dict(kept=A + 2), dict(nl=A + 2)):
        assert evict(lib, **bad) == MISALIGNED, bad


def test_overlapping_outputs(lib):
    """Rows that a call writes must be apart; rows that it only reads may be the same."""
    for bad in (dict(k_stride_page=0), dict(v_stride_slot=0), dict(k_stride_head=120), dict(v_stride_head=0)):
        assert append(lib, **bad) == INVALID, bad
        assert "overlap" in dcp.dcp_last_error()
        assert evict(lib, dst=cache(**bad)) == INVALID, bad
        assert "overlap" in dcp.dcp_last_error()
        assert evict(lib, B=0, **bad) == OK and attend(lib, B=0, **bad) == OK
    # dimensions of one entry
    assert append(lib, R=0, num_pages=1, k_stride_page=0, page_size=1, v_stride_slot=0, heads=1, k_stride_head=0) == OK
    for call, bad in ((weigh, dict(wb=0)), (weigh, dict(wh=63)), (evict, dict(nb=0)), (evict, dict(nh=31)),
                      (attend, dict(logits=A, cap=64, lb=512, lh=63)), (attend, dict(logits=A, cap=64, lb=0, lh=64))):
        assert call(lib, **bad) == INVALID, bad
        assert "overlap" in dcp.dcp_last_error()


def tensors():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    return dict(q=torch.zeros(3, 8, 64, dtype=torch.bfloat16), k=k, v=k.clone(),
                table=torch.zeros(3, 2, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32))


def test_binding_rejects_cpu_tensors():
    t = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        dcp.paged_attention(t["q"], t["k"], t["v"], t["table"], t["lens"])
    with pytest.raises(ValueError, match="CUDA"):
        dcp.dcp_kv_append(t["k"][0, :3], t["v"][0, :3], t["k"], t["v"], t["table"], t["lens"],
                          torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        dcp.dcp_kv_weights(torch.zeros(3, 8, 32), torch.zeros(3, 8), t["lens"], torch.zeros(3, 2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        dcp.kv_evict(torch.zeros(3, 2, 32), t["k"], t["v"], t["table"], t["lens"], t["table"], 8)
    with pytest.raises(dcp.DCPError):
        dcp.kv_evict(torch.zeros(3, 2, 32), t["k"], t["v"], t["table"], t["lens"], t["table"], 0)
    with pytest.raises(ValueError, match="world_size"):
        dcp.paged_attention_pack(t["q"], t["k"], t["v"], t["table"], t["lens"], 3)


# ---- the reference itself -----------------------------------------------------------------------
@pytest.mark.parametrize("n,s", [(1, 1), (2, 1), (3, 4), (8, 16)])
def test_reference_lengths_match_the_formula(n, s):
    for seq in range(0, 200, 7):
        parts = []
        for r in range(n):
            full, rest = divmod(seq, n * s)
            formula = full * s + min(max(rest - r * s, 0), s)
            assert ref.local_len(seq, r, n, s) == formula
            parts.append(formula)
        assert sum(parts) == seq


def test_reference_shards_combine_to_the_whole():
    """Attention over the shards of a request, merged by their LSEs, is attention over all of it,
    and the weights of all shards sum to the group size."""
    g = torch.Generator().manual_seed(3)
    q, k, v = torch.randn(1, 4, 16, generator=g), torch.randn(37, 2, 16, generator=g), torch.randn(37, 2, 16, generator=g)
    out, lse, logits, _, _ = ref.attention(q, [k], [v], 0.25)
    n, s = 3, 4
    acc, total, wsum = np.zeros_like(out), np.zeros_like(lse), np.zeros((1, 2))
    for r in range(n):
        own = ref.owned(37, r, n, s)
        o, l, lo, _, _ = ref.attention(q, [k[own]], [v[own]], 0.25)
        acc += np.exp(l - lse)[..., None] * o
        total += np.exp(l - lse)
        w = ref.weights(np.asarray(lo), lse, np.zeros((1, 2, len(own))), [len(own)], True)
        wsum += w.sum(-1)
    np.testing.assert_allclose(acc, out, atol=1e-12)
    np.testing.assert_allclose(total, 1.0, atol=1e-12)
    np.testing.assert_allclose(wsum, 2.0, atol=1e-12)


def test_reference_selection():
    nan, inf = math.nan, math.inf
    assert ref.select(np.array([1.0, 2.0]), 2, 0) == [0, 1]
    assert ref.select(np.array([1.0, 3.0, 2.0, 0.0]), 2, 1) == [1, 3]
    assert ref.select(np.array([1.0, 1.0, 1.0, 1.0]), 2, 0) == [0, 1]          # ties: lowest position
    assert ref.select(np.array([nan, -inf, nan, 5.0]), 2, 0) == [1, 3]          # NaN below -inf
    assert ref.select(np.array([nan, nan, nan]), 2, 0) == [0, 1]
    assert ref.select(np.array([0.0, 9.0, 9.0]), 2, 2) == [1, 2]

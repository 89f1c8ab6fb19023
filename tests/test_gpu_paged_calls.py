"""Calls of the paged cache that the documentation allows and that lie off the usual path: the same slot
named twice, lengths that name nothing, arrays wider than their content."""
from __future__ import annotations

import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
from decode_context_attention_dcp_b200 import paged

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

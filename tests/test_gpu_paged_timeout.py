"""The paged attention's bounded waits run out on purpose, without faulting or hanging the GPU:
dcp_testing_paged_attention_stalled makes each wait expect 16 bytes that never arrive (every copy still
lands) and give up after 20 ms.  The kernels must return, count each warp that waits once, whatever
the element type, and leave the device usable for the next, right call."""
from __future__ import annotations

import math

import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref
from decode_context_attention_dcp_b200.paged import _cache

pytestmark = pytest.mark.gpu


def stalled(q, k, v, table, seq):
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(dcp.paged_attention_workspace(q, k), dtype=torch.uint8, device="cuda")
    st = dcp.library().dcp_testing_paged_attention_stalled(
        _cache(k, v, table, q.shape[0]), q.data_ptr(), seq.data_ptr(), out.data_ptr(), lse.data_ptr(), q.shape[0],
        q.shape[1], q.stride(0), q.stride(1), 1 / math.sqrt(q.shape[2]), ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert st == 0, dcp.dcp_last_error()
    torch.cuda.synchronize()


# 3 requests of one whole tile for each of 2 key heads, by a cluster of blocks or in even shares: every warp of 6
# blocks waits once.  Then 8 long ones, of which each block of the resident wave gets several tiles.
@pytest.mark.parametrize("dtype,D,tile,warps,resident", [("bf16", 64, 64, 4, 3), ("fp16", 128, 64, 4, 3),
                                                         ("fp32", 64, 64, 4, 3), ("fp32", 256, 48, 3, 2),
                                                         ("bf16", 256, 96, 6, 1)])
@pytest.mark.parametrize("page", [16, 8])
def test_waits_that_run_out_are_counted(dtype, D, tile, warps, resident, page):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for lens, width, want in (([tile] * 3, None, 6 * warps), ([tile] * 3, 700, 6 * warps),
                              ([60 * tile] * 8, 1000, sms * resident * warps)):
        case = ref.PagedCase(lens, 2, D, page, dtype, seed=D, width=width)
        g = torch.Generator().manual_seed(1)
        q = torch.randn(len(lens), 4, D, generator=g).to(ref.DTYPES[dtype]).cuda()
        k, v, table = case.gpu()
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert dcp.dcp_wait_timeouts(reset=True) == 0
        stalled(q, k, v, table, seq)
        assert dcp.dcp_wait_timeouts() == want
        assert dcp.dcp_wait_timeouts(reset=True) == want
        assert dcp.dcp_wait_timeouts() == 0
        out, lse = dcp.paged_attention(q, k, v, table, seq)
        r = ref.attention(q.cpu(), case.keys, case.values, 1 / math.sqrt(D))
        ref.assert_attention(out, lse, r, lens[0], dtype)
        assert dcp.dcp_wait_timeouts() == 0


def test_calls_without_tensor_copies_do_not_wait():
    case = ref.PagedCase([50, 7], 2, 64, 12, "bf16", seed=2)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    k, v, table = case.gpu()
    stalled(q, k, v, table, torch.tensor([50, 7], dtype=torch.int32, device="cuda"))
    assert dcp.dcp_wait_timeouts() == 0

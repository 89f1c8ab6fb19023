"""Paged attention over caches that hold infinities and NaN at positions that count: the values' columns
are what IEEE products with the softmax weights give, all others stay within the usual bounds."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import decode_context_attention_dcp_b200 as dcp
import paged_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# a table wide enough that the tiles are shared evenly over the device instead of a cluster per request
WIDE = 700


def expected_columns(case, q, scale, held_out=()):
    """[B, H, D]: the sum of weight * value over the values that are not finite, 0 where there is none.
    held_out: (request, position) of logit -inf, whose weight is 0."""
    B, H, D = q.shape
    out = np.zeros((B, H, D))
    for b in range(B):
        kk, vv = case.keys[b].double().numpy(), case.values[b].double().numpy()
        for h in range(H):
            j = h // (H // case.heads)
            x = scale * (kk[:, j] @ q[b, h].double().numpy())
            for r, p in held_out:
                if r == b:
                    x[p] = -INF
            if not len(x):
                continue
            w = np.exp(x - x.max())
            with np.errstate(invalid="ignore"):
                for p, col in zip(*np.nonzero(~np.isfinite(vv[:, j]))):
                    out[b, h, col] += w[p] * vv[p, j, col]
    return out


def check(case, H, spots, base_e=True, low=()):
    """spots: (request, position, key head, column, value) written into the values; low: (request,
    position) whose keys get a logit of -inf (element 0, where the query is positive)."""
    B, D, dtype = len(case.lens), case.D, case.dtype
    g = torch.Generator().manual_seed(case.seed + 3)
    q = torch.randn(B, H, D, generator=g).to(ref.DTYPES[dtype])
    q[:, :, 0] = q[:, :, 0].abs() + 0.125
    for b, p, j, col, value in spots:
        case.values[b][p, j, col] = value
        case.v[int(case.table[b, p // case.page]), p % case.page, j, col] = value
    finite = [v.clone() for v in case.values]
    for v in finite:
        v[~torch.isfinite(v)] = 0
    for b, p in low:
        case.k[int(case.table[b, p // case.page]), p % case.page, :, 0] = -INF
    scale = float(np.float32(1 / math.sqrt(D)))
    want = expected_columns(case, q, scale, low)
    held = [[p for p in range(n) if (b, p) not in low] for b, n in enumerate(case.lens)]
    r = ref.attention(q, case.keys, finite, scale, held)
    k, v, table = case.gpu()
    out, lse = Guarded((B, H, D), q.dtype), Guarded((B, H), torch.float32)
    seq = torch.tensor(case.lens, dtype=torch.int32, device="cuda")
    dcp.dcp_paged_attention(q.cuda(), k, v, table, seq, out.tensor, lse.tensor, is_lse_base_on_e=base_e)
    out.check(), lse.check()
    got = out.tensor.cpu().double()
    special = torch.from_numpy(want != 0)
    np.testing.assert_array_equal(got[special].numpy(), want[want != 0])
    got[special] = 0
    r[0][want != 0] = 0
    ref.assert_attention(got, lse.tensor, r, max(case.lens), dtype, base_e)
    send = dcp.paged_attention_pack(q.cuda(), k, v, table, seq, 2, is_lse_base_on_e=base_e)
    packed = dcp.pack(out.tensor, lse.tensor, 2)
    assert torch.equal(send[..., :D].float().nan_to_num(1e9), packed[..., :D].float().nan_to_num(1e9))
    assert torch.equal(send[..., D:].contiguous().view(torch.int32), packed[..., D:].contiguous().view(torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,page", [(64, 16), (80, 24), (128, 5), (256, 16)])
@pytest.mark.parametrize("width", [None, WIDE])
def test_infinite_values(dtype, D, page, width):
    """One position (weight 1), a few, several tiles; one infinity, two of a sign, both signs, NaN."""
    case = ref.PagedCase([1, 3, 40, 0, 150], 2, D, page, dtype, seed=D, width=width)
    spots = [(0, 0, 0, 0, INF), (0, 0, 0, 3, -INF), (0, 0, 1, D - 1, NAN),
             (1, 2, 1, 5, -INF),
             (2, 0, 0, 7, INF), (2, 39, 0, 7, INF), (2, 1, 1, 8, INF), (2, 30, 1, 8, -INF), (2, 17, 0, 9, NAN),
             (4, 149, 0, 0, INF), (4, 64, 1, 2, -INF), (4, 3, 1, 2, -INF), (4, 100, 0, 33, INF), (4, 101, 0, 34, -INF)]
    check(case, 6, spots, base_e=D != 80)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_infinite_values_of_requests_cut_into_parts(dtype):
    """A long request, whose parts are joined, beside short ones that a block finishes."""
    case = ref.PagedCase([5, 9001, 70], 2, 64, 16, dtype, seed=8)
    spots = [(1, 9000, 0, 1, INF), (1, 0, 1, 63, -INF), (1, 4000, 0, 20, INF), (1, 7000, 0, 20, -INF),
             (1, 77, 1, 5, NAN), (0, 4, 1, 2, INF), (2, 69, 0, 2, -INF)]
    check(case, 16, spots)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("width", [None, WIDE])
def test_infinite_values_at_logits_of_minus_infinity(dtype, width):
    """0 times an infinity is NaN; finite values add nothing there."""
    case = ref.PagedCase([20, 50], 2, 64, 16, dtype, seed=9, width=width)
    check(case, 4, [(0, 3, 0, 5, INF), (0, 4, 1, 6, INF), (1, 49, 1, 7, -INF)], low=[(0, 3), (1, 49), (1, 20)])


@pytest.mark.parametrize("H,heads,D", [(40, 1, 128), (33, 1, 64), (20, 1, 256)])
def test_infinite_values_of_wide_groups(H, heads, D):
    """Several blocks of heads per key head, in one call with 700 requests whose blocks finish many each."""
    case = ref.PagedCase([70, 0, 129, 16], heads, D, 16, "bf16", seed=H)
    check(case, H + H % 2, [(0, 69, 0, 0, INF), (2, 64, 0, 50, -INF), (3, 0, 0, 1, NAN)])


def test_infinite_values_of_many_requests():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 60, (900,), generator=g).tolist()
    spots = [(b, n - 1, b % 2, b % 64, INF if b % 3 else -INF) for b, n in enumerate(lens) if n and b % 5 == 0]
    check(ref.PagedCase(lens, 2, 64, 16, "bf16", seed=5), 4, spots)


def test_a_cache_of_infinite_values():
    """Every value infinite: every column is, and the call still ends soon."""
    case = ref.PagedCase([3000, 64], 1, 64, 16, "bf16", seed=6)
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    k, v, table = case.gpu()
    v = torch.full_like(v, -INF)
    out, lse = dcp.paged_attention(q.cuda(), k, v, table, torch.tensor([3000, 64], dtype=torch.int32, device="cuda"))
    assert (out == -INF).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("width", [None, WIDE])
def test_fp32_keys_and_values_next_to_the_largest(width):
    """fp32 factors that round to infinity as tf32 make NaN of their row (keys) or column (values)."""
    case = ref.PagedCase([40, 40], 1, 64, 16, "fp32", seed=7, width=width)
    top = torch.finfo(torch.float32).max
    case.k[int(case.table[0, 0]), 3, 0, 5] = top
    case.v[int(case.table[1, 0]), 3, 0, 5] = -top
    k, v, table = case.gpu()
    q = torch.ones(2, 2, 64, device="cuda")
    out, lse = dcp.paged_attention(q, k, v, table, torch.tensor([40, 40], dtype=torch.int32, device="cuda"))
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isnan(out[1, :, 5]).all() and torch.isfinite(lse[1]).all()
    assert torch.isfinite(out[1, :, :5]).all() and torch.isfinite(out[1, :, 6:]).all()

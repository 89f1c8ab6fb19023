"""Which outputs of the paged calls are refused because rows share elements, against a count of the elements."""
from __future__ import annotations

import random

import pytest

import decode_context_attention_dcp_b200 as dcp
from test_paged_refusals import INVALID, append, attend, cache, evict, weigh


@pytest.fixture(scope="module")
def lib():
    return dcp.library()


def overlap(n, s, width):
    seen = set()
    for i in range(n[0]):
        for j in range(n[1]):
            for k in range(n[2]):
                row = range(i * s[0] + j * s[1] + k * s[2], i * s[0] + j * s[1] + k * s[2] + width)
                if not seen.isdisjoint(row):
                    return True
                seen.update(row)
    return False


def test_against_a_count(lib):
    rng = random.Random(5)
    found = [0, 0]
    for _ in range(4000):
        n = [rng.randint(1, 5) for _ in range(3)]
        width = rng.randint(1, 4)
        s = [rng.choice([0, width, 2 * width, 3 * width, rng.randint(0, 40)]) for _ in range(3)]
        want = overlap(n, s, width)
        assert lib.dcp_testing_rows_overlap(*n, *s, width) == want, (n, s, width)
        found[want] += 1
    assert min(found) > 300  # both kinds are met


def test_large_layouts_are_accepted(lib):
    """Pools of the usual layouts, of any size, and strides next to the 64-bit limit."""
    D = 128
    for n in ((1 << 24, 16, 8), (1 << 20, 4096, 1), (3, 1 << 20, 64)):
        pages, slots, heads = n
        for s in ((slots * heads * D, heads * D, D), (slots * heads * D, D, slots * D),
                  (2 * slots * heads * D, heads * D, D), (heads * D, pages * heads * D, D)):
            assert lib.dcp_testing_rows_overlap(*n, *s, D) == 0, (n, s)
    assert lib.dcp_testing_rows_overlap(2, 2, 1, 1 << 62, (1 << 62) - 1, 0, 8) == 1
    assert lib.dcp_testing_rows_overlap(2, 2, 1, 1 << 62, 1 << 40, 0, 8) == 0


def test_rows_that_lie_inside_one_another_are_refused(lib):
    """Strides of at least a row under which rows of two dimensions, or of three, still meet."""
    for call, bad in ((weigh, dict(wb=64, wh=64)), (evict, dict(nb=32, nh=32)), (evict, dict(nb=40, nh=32)),
                      (attend, dict(logits=0x10000, cap=64, lb=64, lh=64)),
                      (attend, dict(logits=0x10000, cap=64, lb=128, lh=64))):
        assert call(lib, **bad) == INVALID, bad
        assert "overlap" in dcp.dcp_last_error()
    # pages that begin inside the one before: at a slot of it, and at its last slot's second head
    for bad in (dict(k_stride_page=8 * 256), dict(v_stride_page=15 * 256 + 128), dict(k_stride_slot=128)):
        assert append(lib, **bad) == INVALID, bad
        assert "overlap" in dcp.dcp_last_error()
        assert evict(lib, dst=cache(**bad)) == INVALID, bad

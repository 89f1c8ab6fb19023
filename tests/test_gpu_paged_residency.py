"""The paged attention's grid is one resident wave: every kernel has as many blocks on an SM as its launch and
its workspace count on."""
from __future__ import annotations

import ctypes

import pytest

import decode_context_attention_dcp_b200 as dcp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8, 16, 33])
@pytest.mark.parametrize("page", [16, 8, 5])
@pytest.mark.parametrize("cluster", [0, 1])
def test_one_resident_wave(dtype, head_dim, group, page, cluster):
    out = (ctypes.c_int32 * 2)()
    assert dcp.library().dcp_testing_paged_attention_resident(group, head_dim, dtype, page, cluster, out) == 0
    assert out[0] >= out[1] >= 1, (out[0], out[1])

"""Host-side edges of the 4-bit cache's C ABI; no GPU needed."""
import ctypes

import pytest

import sparse_attention_indexer_stable_gb300 as dk

from .test_kv4_capi import attention, cache


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("name", ["softcap", "scale"])
def test_a_scale_or_cap_that_is_not_finite_is_refused(name, value):
    args = attention(**{name: value})
    assert dk.library().dcp_kv4_attention(cache(), args, None) == dk.DCP_ERR_INVALID
    n = ctypes.c_size_t(7)
    assert dk.library().dcp_kv4_attention_workspace_size(
        cache(), args, ctypes.byref(n)) == dk.DCP_ERR_INVALID

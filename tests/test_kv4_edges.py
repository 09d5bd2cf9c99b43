"""Host-side edges of the 4-bit cache's C ABI; no GPU needed."""
import ctypes
import sysconfig

import pytest

import sparse_attention_indexer_stable_gb300 as dk
from sparse_attention_indexer_stable_gb300 import _build

from .test_kv4_capi import attention, cache


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("name", ["softcap", "scale"])
def test_a_scale_or_cap_that_is_not_finite_is_refused(name, value):
    args = attention(**{name: value})
    assert dk.library().dcp_kv4_attention(cache(), args, None) == dk.DCP_ERR_INVALID
    n = ctypes.c_size_t(7)
    assert dk.library().dcp_kv4_attention_workspace_size(
        cache(), args, ctypes.byref(n)) == dk.DCP_ERR_INVALID


@pytest.mark.parametrize("with_ids", [False, True])
@pytest.mark.parametrize("heads,group,rows,width", [
    (65536, 1, 2 ** 31 - 1, 2 ** 22), (65536, 16384, 2 ** 20, 2 ** 22), (1, 1, 2 ** 31 - 1, 2 ** 23),
    (65536, 32767, 2 ** 31 - 1, 1), (2, 4, 2 ** 28, 2 ** 23 - 1)])
def test_sizes_whose_products_pass_64_bits_are_refused(heads, group, rows, width, with_ids):
    """Refused before they are multiplied any further (a build with the
    compiler's overflow checks reports nothing)."""
    c = cache(heads=heads, dim=256, page=256, pages=8)
    n = ctypes.c_size_t(7)
    args = attention(rows=rows, num_seqs=rows, q_heads=heads * group, table_width=width,
                     ids=16 if with_ids else 0, num_ids=2 ** 31 - 1 if with_ids else 0)
    assert dk.library().dcp_kv4_attention_workspace_size(
        c, args, ctypes.byref(n)) == dk.DCP_ERR_UNSUPPORTED
    assert n.value == 7


def test_the_binding_is_built_for_one_python_and_one_torch(monkeypatch):
    """Another Python, torch or CUDA of torch: another file, not one of the
    wrong ABI."""
    torch = pytest.importorskip("torch")
    paths = {_build.binding_path()}
    with monkeypatch.context() as m:
        real = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var",
                  lambda name: ".cpython-399-none.so" if name == "EXT_SUFFIX" else real(name))
        paths.add(_build.binding_path())
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0")
        paths.add(_build.binding_path())
    with monkeypatch.context() as m:
        m.setattr(torch.version, "cuda", "1.0")
        paths.add(_build.binding_path())
    assert len(paths) == 4 and all(p.endswith(".so") for p in paths)

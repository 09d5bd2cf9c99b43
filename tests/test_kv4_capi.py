"""Host-side checks of the 4-bit cache's C ABI and of its reference in 64
bits; no GPU needed."""
import ctypes

import numpy as np
import pytest

import sparse_attention_indexer_stable_gb300 as dk
from sparse_attention_indexer_stable_gb300 import kv4

from . import kv4_reference as ref

FAKE = 0x1000  # never dereferenced: every case below fails validation first


def cache(ptr=FAKE, pages=8, page=16, heads=2, dim=128, ku=1.0, vu=1.0):
    return kv4._CACHE.pack(ptr, ptr, ptr, ptr, pages, page, heads, dim, ku, vu)


def attention(**change):
    a = dict(q=FAKE, q_row=1024, q_head=128, table=FAKE, table_stride=4, lens=FAKE, starts=0,
             owner=0, ids=0, ids_stride=0, row_starts=0, weights=0, w_stride=0, w_width=0,
             out=FAKE, lse=FAKE, workspace=0, workspace_bytes=0, dtype=dk.DCP_BF16, rows=3,
             q_heads=8, num_seqs=3, table_width=4, num_ids=0, max_len=0, scale=0.0, softcap=0.0)
    assert set(change) <= set(a)
    a.update(change)
    return kv4._ATTENTION.pack(*a.values())


def evict(**change):
    a = dict(table=FAKE, table_stride=4, lens=FAKE, weights=FAKE, w_stride=64, out_table=FAKE,
             out_stride=1, kept=FAKE, out_lens=FAKE, out_weights=FAKE, num_seqs=3, table_width=4,
             w_width=64, budget=16, sinks=0, recent=0)
    assert set(change) <= set(a)
    a.update(change)
    return kv4._EVICT.pack(*a.values())


BAD_CACHES = [
    (dict(ptr=0), dk.DCP_ERR_INVALID), (dict(ptr=0x1008), dk.DCP_ERR_INVALID),
    (dict(pages=-1), dk.DCP_ERR_INVALID), (dict(page=0), dk.DCP_ERR_INVALID),
    (dict(heads=0), dk.DCP_ERR_INVALID), (dict(ku=0.75), dk.DCP_ERR_INVALID),
    (dict(vu=0.0), dk.DCP_ERR_INVALID), (dict(vu=float("inf")), dk.DCP_ERR_INVALID),
    (dict(page=24), dk.DCP_ERR_UNSUPPORTED), (dict(page=1 << 17), dk.DCP_ERR_UNSUPPORTED),
    (dict(dim=96), dk.DCP_ERR_UNSUPPORTED), (dict(pages=1 << 28), dk.DCP_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_every_call_checks_the_cache(change, want):
    lib, c = dk.library(), cache(**change)
    assert lib.dcp_kv4_append(c, FAKE, FAKE, dk.DCP_F16, 1, 0, 0, 0, 0, FAKE, None) == want
    assert lib.dcp_kv4_read(c, FAKE, FAKE, dk.DCP_F16, 1, FAKE, None) == want
    assert lib.dcp_kv4_attention(c, attention(), None) == want
    assert lib.dcp_kv4_evict(c, evict(), None) == want
    n = ctypes.c_size_t(7)
    assert lib.dcp_kv4_attention_workspace_size(c, attention(), ctypes.byref(n)) == want


@pytest.mark.parametrize("args,want", [
    ((FAKE, FAKE, 3, 1), dk.DCP_ERR_INVALID), ((FAKE, FAKE, dk.DCP_F32, -1), dk.DCP_ERR_INVALID),
    ((0, FAKE, dk.DCP_F32, 1), dk.DCP_ERR_INVALID), ((FAKE, 0, dk.DCP_F32, 1), dk.DCP_ERR_INVALID),
    ((FAKE, FAKE, dk.DCP_F32, 1 << 40), dk.DCP_ERR_UNSUPPORTED), ((0, 0, dk.DCP_F32, 0), dk.DCP_OK),
])
def test_store_argument_errors(args, want):
    k, v, dtype, n = args
    lib = dk.library()
    assert lib.dcp_kv4_append(cache(), k, v, dtype, n, 0, 0, 0, 0, FAKE, None) == want
    assert lib.dcp_kv4_read(cache(), k, v, dtype, n, FAKE, None) == want
    if n > 0:
        assert lib.dcp_kv4_append(cache(), k, v, dtype, n, 0, 0, 0, 0, None, None) in (
            want, dk.DCP_ERR_INVALID)


def test_read_wants_aligned_outputs():
    assert dk.library().dcp_kv4_read(cache(), FAKE + 8, FAKE, dk.DCP_F16, 1, FAKE,
                                     None) == dk.DCP_ERR_INVALID


@pytest.mark.parametrize("change,want", [
    (dict(dtype=dk.DCP_F32), dk.DCP_ERR_INVALID), (dict(rows=-1), dk.DCP_ERR_INVALID),
    (dict(q_heads=7), dk.DCP_ERR_INVALID), (dict(q_heads=0), dk.DCP_ERR_INVALID),
    (dict(num_seqs=2), dk.DCP_ERR_INVALID), (dict(table_width=-1), dk.DCP_ERR_INVALID),
    (dict(max_len=-1), dk.DCP_ERR_INVALID), (dict(ids=FAKE, num_ids=-1), dk.DCP_ERR_INVALID),
    (dict(softcap=-1.0), dk.DCP_ERR_INVALID), (dict(softcap=float("nan")), dk.DCP_ERR_INVALID),
    (dict(weights=FAKE, owner=FAKE), dk.DCP_ERR_INVALID), (dict(w_width=-1), dk.DCP_ERR_INVALID),
    (dict(q=0), dk.DCP_ERR_INVALID), (dict(lens=0), dk.DCP_ERR_INVALID),
    (dict(table=0), dk.DCP_ERR_INVALID), (dict(out=0), dk.DCP_ERR_INVALID),
    (dict(lse=0), dk.DCP_ERR_INVALID), (dict(out=FAKE + 2), dk.DCP_ERR_INVALID),
    (dict(weights=FAKE), dk.DCP_ERR_INVALID),           # no workspace
    (dict(weights=FAKE, workspace=FAKE, workspace_bytes=64), dk.DCP_ERR_INVALID),
    (dict(table_width=1 << 28), dk.DCP_ERR_UNSUPPORTED),
    (dict(weights=FAKE, q_heads=4098), dk.DCP_ERR_UNSUPPORTED),
    (dict(rows=0, q=0, lens=0, out=0, lse=0), dk.DCP_OK),
])
def test_attention_argument_errors(change, want):
    assert dk.library().dcp_kv4_attention(cache(), attention(**change), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(num_seqs=-1), dk.DCP_ERR_INVALID), (dict(budget=0), dk.DCP_ERR_INVALID),
    (dict(sinks=-1), dk.DCP_ERR_INVALID), (dict(recent=-1), dk.DCP_ERR_INVALID),
    (dict(sinks=9, recent=8), dk.DCP_ERR_INVALID), (dict(w_width=-1), dk.DCP_ERR_INVALID),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dk.DCP_ERR_INVALID),
    (dict(table=0), dk.DCP_ERR_INVALID), (dict(lens=0), dk.DCP_ERR_INVALID),
    (dict(weights=0), dk.DCP_ERR_INVALID), (dict(out_table=0), dk.DCP_ERR_INVALID),
    (dict(kept=0), dk.DCP_ERR_INVALID), (dict(out_lens=0), dk.DCP_ERR_INVALID),
    (dict(out_weights=0), dk.DCP_ERR_INVALID), (dict(table_width=1 << 28), dk.DCP_ERR_UNSUPPORTED),
    (dict(num_seqs=0, table=0, lens=0, weights=0), dk.DCP_OK),
])
def test_evict_argument_errors(change, want):
    assert dk.library().dcp_kv4_evict(cache(), evict(**change), None) == want


def test_null_arguments():
    lib = dk.library()
    assert lib.dcp_kv4_attention(None, attention(), None) == dk.DCP_ERR_INVALID
    assert lib.dcp_kv4_attention(cache(), None, None) == dk.DCP_ERR_INVALID
    assert lib.dcp_kv4_evict(cache(), None, None) == dk.DCP_ERR_INVALID
    assert lib.dcp_kv4_attention_workspace_size(cache(), attention(), None) == dk.DCP_ERR_INVALID


def test_the_binding_loads_and_refuses_what_is_no_cache():
    """The torch side is built against this torch and connected to the library."""
    binding = kv4._bind()
    with pytest.raises(TypeError):
        binding.append(b"", 0, None, None, None, None)
    with pytest.raises(TypeError):
        binding.append(cache())
    for call in (lambda: dk.kv4_append(None, None, None, None), lambda: dk.kv4_read(None, None),
                 lambda: dk.kv4_attention(None, None, None, None),
                 lambda: dk.kv4_evict(None, None, None, None, None, 1)):
        with pytest.raises(TypeError):
            call()


def test_reference_grid_and_rounding():
    """The reference's own arithmetic: grid values, ties to even, saturation."""
    assert ref.SCALES[1] == 2.0 ** -9 and ref.SCALES[126] == 448 and ref.SCALES[56] == 1.0
    assert np.all(np.diff(ref.SCALES) > 0)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e9])
    assert ref.MAGNITUDES[ref.nearest(ties, ref.MAGNITUDES)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    x = np.random.default_rng(0).standard_normal((4, 64))
    codes, scales = ref.encode(x)
    y = ref.decode(ref.pack(codes), scales)
    # half of the widest step (2) of the largest scale, which rounds by 1/16
    amax = np.abs(x).reshape(4, 4, 16).max(-1).repeat(16, -1)
    assert np.all(np.abs(x - y) <= amax / 6 * 1.0625 * 1.0 + amax * 0.0625)


def test_reference_attention_against_a_hand_worked_row():
    """Two tokens, equal scores: the mean of their values; the cap and the
    weights by hand."""
    H, D = 1, 64
    k = np.zeros((1, 2, H, D))
    v = np.zeros((1, 2, H, D))
    v[0, 0], v[0, 1] = 6.0, -3.0
    planes = []
    for x in (k, v):
        c, s = ref.encode(x)
        planes.append((ref.pack(c), s))
    planes = (planes[0][0], planes[1][0], planes[0][1], planes[1][1])
    out, lse, w, *_ = ref.attention(planes, np.ones((1, 2, D)), np.zeros((1, 1), int), [2],
                                    softcap=5.0, positions=2)
    assert np.allclose(out, 1.5) and np.allclose(lse, np.log(2)) and np.allclose(w, 1.0)


def test_reference_eviction_by_hand():
    w = np.array([0, 3, 1, 3, 2, np.nan, 9, 0])
    assert ref.evict(8, w, 4, 1, 1).tolist() == [0, 1, 6, 7]
    assert ref.evict(8, w, 3, 0, 0).tolist() == [1, 3, 6]
    assert ref.evict(3, w, 4, 1, 1).tolist() == [0, 1, 2]
    assert ref.evict(7, w, 6, 0, 0).tolist() == [0, 1, 2, 3, 4, 6]

"""Host-side checks of the C ABI of prompts and of a batch's bookkeeping, and of
their references; no GPU needed."""
import ctypes
import struct

import numpy as np
import pytest

import sparse_attention_indexer_stable_gb300 as dk

from . import prompt_reference as ref

FAKE = 0x1000  # never dereferenced: every case below fails validation first

EXTEND = struct.Struct("Pq11Pqiiiii4x")
ROTARY = struct.Struct("4P8qPPqiiiiiif4x")
PROMPT = struct.Struct("3P6qPPPqiiiiiiiff4x")


def extend(**change):
    a = dict(table=FAKE, table_stride=4, lens=FAKE, counts=FAKE, free=FAKE, used=FAKE, slots=FAKE,
             positions=FAKE, owner=FAKE, row_lens=FAKE, starts=FAKE, out_lens=FAKE, out_used=FAKE,
             num_pages=8, page_size=16, num_seqs=3, table_width=4, num_free=5, places=7)
    assert set(change) <= set(a)
    a.update(change)
    return EXTEND.pack(*a.values())


def rotary(**change):
    a = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, q_row=512, q_head=128, k_row=128, k_head=128,
             qo_row=512, qo_head=128, ko_row=128, ko_head=128, positions=FAKE, turns=FAKE, tokens=2,
             dtype=dk.DCP_BF16, q_heads=4, k_heads=1, dim=128, turned=64, interleaved=0,
             magnitude=1.0)
    assert set(change) <= set(a)
    a.update(change)
    return ROTARY.pack(*a.values())


def prompt(**change):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_row=512, q_head=128, k_row=128, k_head=128, v_row=128,
             v_head=128, starts=FAKE, out=FAKE, lse=FAKE, rows=3, dtype=dk.DCP_BF16, q_heads=4,
             kv_heads=1, dim=128, num_seqs=1, causal=1, window=0, scale=0.0, softcap=0.0)
    assert set(change) <= set(a)
    a.update(change)
    return PROMPT.pack(*a.values())


@pytest.mark.parametrize("change,want", [
    (dict(num_pages=-1), dk.DCP_ERR_INVALID), (dict(page_size=0), dk.DCP_ERR_INVALID),
    (dict(num_seqs=-1), dk.DCP_ERR_INVALID), (dict(table_width=-1), dk.DCP_ERR_INVALID),
    (dict(num_free=-1), dk.DCP_ERR_INVALID), (dict(places=-1), dk.DCP_ERR_INVALID),
    (dict(table=0), dk.DCP_ERR_INVALID), (dict(lens=0), dk.DCP_ERR_INVALID),
    (dict(counts=0), dk.DCP_ERR_INVALID), (dict(free=0), dk.DCP_ERR_INVALID),
    (dict(used=0), dk.DCP_ERR_INVALID), (dict(slots=0), dk.DCP_ERR_INVALID),
    (dict(positions=0), dk.DCP_ERR_INVALID), (dict(owner=0), dk.DCP_ERR_INVALID),
    (dict(row_lens=0), dk.DCP_ERR_INVALID), (dict(starts=0), dk.DCP_ERR_INVALID),
    (dict(out_lens=0), dk.DCP_ERR_INVALID), (dict(out_used=0), dk.DCP_ERR_INVALID),
    (dict(page_size=24), dk.DCP_ERR_UNSUPPORTED), (dict(page_size=1 << 17), dk.DCP_ERR_UNSUPPORTED),
    (dict(num_seqs=16385), dk.DCP_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 28), dk.DCP_ERR_UNSUPPORTED),
    (dict(table_width=1 << 27), dk.DCP_ERR_UNSUPPORTED),
])
def test_extend_argument_errors(change, want):
    assert dk.library().dcp_kv4_extend(extend(**change), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=3), dk.DCP_ERR_INVALID), (dict(tokens=-1), dk.DCP_ERR_INVALID),
    (dict(q_heads=-1), dk.DCP_ERR_INVALID), (dict(k_heads=-1), dk.DCP_ERR_INVALID),
    (dict(turned=0), dk.DCP_ERR_INVALID), (dict(turned=3), dk.DCP_ERR_INVALID),
    (dict(turned=130), dk.DCP_ERR_INVALID), (dict(magnitude=float("nan")), dk.DCP_ERR_INVALID),
    (dict(q=0), dk.DCP_ERR_INVALID), (dict(q_out=0), dk.DCP_ERR_INVALID),
    (dict(k=0), dk.DCP_ERR_INVALID), (dict(k_out=0), dk.DCP_ERR_INVALID),
    (dict(positions=0), dk.DCP_ERR_INVALID), (dict(turns=0), dk.DCP_ERR_INVALID),
    (dict(dim=1026), dk.DCP_ERR_UNSUPPORTED), (dict(q_heads=65537), dk.DCP_ERR_UNSUPPORTED),
    (dict(k_heads=65537), dk.DCP_ERR_UNSUPPORTED), (dict(tokens=1 << 31), dk.DCP_ERR_UNSUPPORTED),
    (dict(tokens=0, q=0, k=0, positions=0), dk.DCP_OK), (dict(q_heads=0, k_heads=0), dk.DCP_OK),
])
def test_rotary_argument_errors(change, want):
    assert dk.library().dcp_rotary(rotary(**change), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=dk.DCP_F32), dk.DCP_ERR_INVALID), (dict(rows=-1), dk.DCP_ERR_INVALID),
    (dict(num_seqs=-1), dk.DCP_ERR_INVALID), (dict(q_heads=0), dk.DCP_ERR_INVALID),
    (dict(kv_heads=0), dk.DCP_ERR_INVALID), (dict(kv_heads=3), dk.DCP_ERR_INVALID),
    (dict(window=-1), dk.DCP_ERR_INVALID), (dict(scale=float("inf")), dk.DCP_ERR_INVALID),
    (dict(softcap=float("nan")), dk.DCP_ERR_INVALID), (dict(softcap=-1.0), dk.DCP_ERR_INVALID),
    (dict(q=0), dk.DCP_ERR_INVALID), (dict(k=0), dk.DCP_ERR_INVALID),
    (dict(v=0), dk.DCP_ERR_INVALID), (dict(starts=0), dk.DCP_ERR_INVALID),
    (dict(out=0), dk.DCP_ERR_INVALID), (dict(lse=0), dk.DCP_ERR_INVALID),
    (dict(out=FAKE + 2), dk.DCP_ERR_INVALID), (dict(dim=96), dk.DCP_ERR_UNSUPPORTED),
    (dict(rows=1 << 30), dk.DCP_ERR_UNSUPPORTED), (dict(rows=1 << 40), dk.DCP_ERR_UNSUPPORTED),
    (dict(q=FAKE + 2), dk.DCP_ERR_UNSUPPORTED), (dict(k_row=132), dk.DCP_ERR_UNSUPPORTED),
    (dict(v_row=0), dk.DCP_ERR_UNSUPPORTED), (dict(q_head=-8), dk.DCP_ERR_UNSUPPORTED),
    (dict(q_row=1 << 39), dk.DCP_ERR_UNSUPPORTED),
    (dict(rows=0, q=0, k=0, out=0), dk.DCP_OK), (dict(num_seqs=0), dk.DCP_OK),
])
def test_prompt_argument_errors(change, want):
    assert dk.library().dcp_prompt_attention(prompt(**change), None) == want


def test_null_arguments_and_the_structs_sizes():
    lib = dk.library()
    assert lib.dcp_kv4_extend(None, None) == dk.DCP_ERR_INVALID
    assert lib.dcp_rotary(None, None) == dk.DCP_ERR_INVALID
    assert lib.dcp_prompt_attention(None, None) == dk.DCP_ERR_INVALID
    assert (EXTEND.size, ROTARY.size, PROMPT.size) == (136, 152, 144)


def test_python_refuses_what_is_no_tensor():
    with pytest.raises(TypeError):
        dk.kv4_extend(None, None, None, None, None, 1, 16, 1)
    with pytest.raises(TypeError):
        dk.rotary(None, None, None)
    with pytest.raises(TypeError):
        dk.prompt_attention(None, None, None, None)


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=3), dict(dim=2048), dict(dim=4, base=0.5), dict(dim=4, factor=0.0),
    dict(dim=4, factor=float("inf")), dict(dim=4, original=-1), dict(dim=4, slow=2.0, fast=2.0),
    dict(dim=4, frequencies=[1.0]), dict(dim=4, frequencies=[1.0, float("nan")]),
    dict(dim=4, magnitude=float("inf")), dict(dim=4, device="cpu"),
])
def test_rotary_handle_refusals(kw):
    with pytest.raises(ValueError):
        dk.Rotary(**kw)


def test_reference_extend_by_hand():
    """Two sequences, pages of 2: the first fills its page and takes page 5, the
    second takes page 6 and finds the list empty."""
    got = ref.extend([[3, -1], [-1, -1]], [1, 0], [2, 4], [9, 5, 6], 1, 8, 2, 7)
    assert got[0] == [7, 10, 12, 13, -1, -1, -1, -1]
    assert got[1] == [1, 2, 0, 1, 2, 3, 0, 0] and got[2] == [0, 0, 1, 1, 1, 1, -1, -1]
    assert got[3] == [2, 3, 1, 2, 3, 4, 0, 0]
    assert got[4:7] == ([0, 2, 6], [3, 4], [4]) and got[7] == [[3, 5], [6, -1]]


def test_reference_turn_by_hand():
    x = np.array([[[1.0, 2.0, 3.0]]])
    quarter = [float(ref.TURN / 4)]  # a quarter of a turn a position
    assert np.allclose(ref.turned(x, [1], quarter), [[[-2.0, 1.0, 3.0]]])
    assert np.allclose(ref.turned(x, [2], quarter, magnitude=2.0), [[[-2.0, -4.0, 3.0]]])
    assert np.allclose(ref.turned(x, [-1], quarter, interleaved=True), [[[2.0, -1.0, 3.0]]])


def test_reference_attention_by_hand():
    """Equal scores: row i's output is the mean of what it sees."""
    torch = pytest.importorskip("torch")
    q = torch.zeros(5, 2, 4)
    v = torch.arange(5.0).view(5, 1, 1).expand(5, 1, 4)
    out, lse, _, _ = ref.attention(q, torch.ones(5, 1, 4), v, [0, 3, 5])
    assert torch.allclose(out[:, 1, 0], torch.tensor([0, .5, 1, 3, 3.5]).double())
    assert torch.allclose(lse[:, 0], torch.log(torch.tensor([1, 2, 3, 1, 2.])).double())
    out, _, _, _ = ref.attention(q, torch.ones(5, 1, 4), v, [1, 5], causal=False, window=2)
    assert torch.isnan(out[0]).all() and out[1:, 0, 0].tolist() == [2.5, 2.5, 3.0, 3.5]

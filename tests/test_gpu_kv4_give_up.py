"""A copy that never lands, in attention by runs of a page: the CTA that waits
for it gives up once, reports it, and leaves NaN for what it had not finished;
everything else is right.

The race-check build of the library leaves a tile out when it is told to: it is
neither copied nor armed, so the waits for it run out (after about 2 ms there),
and nothing faults.
"""
import ctypes
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from sparse_attention_indexer_stable_gb300 import _build, kv4  # noqa: E402

from .test_gpu_kv4 import dk, fill, i32, query  # noqa: E402,F401

pytestmark = pytest.mark.gpu

TILE, BEGIN = 32, 2  # tokens of a tile; places that a unit's beginning takes
SHARES = 304


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(_build.build_race_check())
    P = ctypes.c_void_p
    lib.dcp_kv4_attention_workspace_size.argtypes = [P, P, ctypes.POINTER(ctypes.c_size_t)]
    lib.dcp_kv4_attention.argtypes = [P, P, P]
    lib.dcp_topk_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.dcp_kv4_selftest_withhold.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.dcp_kv4_selftest_withhold.restype = None
    yield lib
    lib.dcp_kv4_selftest_withhold(-1, -1)


def attend(lib, cache, q, table, lens):
    """One call through the C ABI; (out, lse, the device's status)."""
    rows, heads, dim = q.shape
    out = torch.empty_like(q)
    lse = torch.empty(rows, heads, device=q.device)
    sizes = dict(dtype=0, rows=rows, q_heads=heads, num_seqs=rows, table_width=table.shape[1],
                 num_ids=0, max_len=0, scale=0.0, softcap=0.0)

    def args(space, n):
        return kv4._ATTENTION.pack(q.data_ptr(), q.stride(0), q.stride(1), table.data_ptr(),
                                   table.stride(0), lens.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0,
                                   out.data_ptr(), lse.data_ptr(), space, n, *sizes.values())

    need = ctypes.c_size_t(0)
    assert lib.dcp_kv4_attention_workspace_size(cache._raw, args(0, 0), ctypes.byref(need)) == 0
    assert need.value > 0  # shares
    space = torch.empty(need.value, dtype=torch.uint8, device=q.device)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.dcp_kv4_attention(cache._raw, args(space.data_ptr(), need.value), stream) == 0
    status = ctypes.c_uint(0)
    assert lib.dcp_topk_device_status(ctypes.byref(status)) == 0  # waits for the device
    return out, lse, status.value


def rows_of_share(share, withheld, tiles, rows, of):
    """The rows that a share walks, and those of them from the one on whose tiles
    hold the group's `withheld`-th tile."""
    total = rows * (BEGIN + tiles)
    per = -(-total // SHARES)
    x, end, walked, all_rows, lost = share * per, min(total, (share + 1) * per), 0, [], []
    while x < end:
        t, at = divmod(x, BEGIN + tiles)
        to = min(BEGIN + tiles, at + end - x)
        here = max(0, to - BEGIN) - max(0, at - BEGIN)
        if here:
            all_rows.append(t)
            if walked + -(-here // of) > withheld:
                lost.append(t)
            walked += -(-here // of)
        x += to - at
    return all_rows, lost


@pytest.mark.parametrize("heads,dim,group,rows,tiles,share,withheld", [
    (8, 64, 2, 304, 20, 7, 5),    # a share is a row
    (8, 128, 2, 608, 10, 300, 13),  # two rows, the second one lost
    (8, 128, 1, 608, 10, 11, 2),  # the first one, and with it the second
    (8, 64, 9, 100, 65, 20, 0),   # a piece of a row, joined with others
    (4, 128, 3, 608, 20, 40, 13),  # two groups of warps, which add up
])
def test_a_copy_that_never_lands(lib, dk, heads, dim, group, rows, tiles, share,  # noqa: F811
                                 withheld):
    rng = np.random.default_rng(rows + tiles)
    page = 16
    cache, _ = fill(dk, rng, 60, page, heads, dim)
    width = tiles * TILE // page
    table = i32(rng.integers(0, 60, (rows, width)))
    lens = i32(np.full(rows, tiles * TILE))
    q, _ = query(rng, rows, heads * group, dim, "f16")
    want_out, want_lse = dk.kv4_attention(cache, q, table, lens)

    lib.dcp_kv4_selftest_withhold(-1, -1)
    out, lse, status = attend(lib, cache, q, table, lens)
    assert status == 0 and torch.equal(out, want_out) and torch.equal(lse, want_lse)

    walked, lost = rows_of_share(share, withheld, tiles, rows, 8 // heads)
    assert lost and len(walked) <= 3
    lib.dcp_kv4_selftest_withhold(share, withheld)
    torch.cuda.synchronize()
    start = time.perf_counter()
    out, lse, status = attend(lib, cache, q, table, lens)
    took = time.perf_counter() - start
    # one wait and the time before the end, 2 ms each; not one for each tile
    assert status == dk.DCP_DEVICE_COPY_TIMEOUT
    assert took < 0.1
    assert torch.isnan(out[lost]).all() and torch.isnan(lse[lost]).all()
    right = np.setdiff1d(np.arange(rows), lost)
    assert torch.equal(out[right], want_out[right]) and torch.equal(lse[right], want_lse[right])

    lib.dcp_kv4_selftest_withhold(-1, -1)
    out, lse, status = attend(lib, cache, q, table, lens)
    assert status == 0 and torch.equal(out, want_out) and torch.equal(lse, want_lse)

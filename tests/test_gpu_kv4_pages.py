"""Attention over ranges by runs of a page: walks that refill the stages many
times, against the definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_kv4 import check, dk, fill, i32, query  # noqa: E402,F401

pytestmark = pytest.mark.gpu

TILE, BEGIN = 32, 2  # tokens of a tile; places that a unit's beginning takes
STAGES = 3


def walk(rng, pages, page, rows, longest, few):
    """A ragged batch whose rows share the cache's pages: (table, lens), a few
    of the rows of nothing and a few of the longest."""
    table = np.stack([rng.permutation(np.resize(np.arange(pages), longest // page))
                      for _ in range(rows)])
    lens = rng.integers(1, longest + 1, rows)
    lens[rng.choice(rows, few, replace=False)] = 0
    lens[rng.choice(np.flatnonzero(lens), few, replace=False)] = longest
    return table, lens


def tiles_of_a_group(heads, dim, group, lens):
    """Tiles that each group of warps walks in a full share."""
    columns = 16 if group > 8 and dim <= 128 else 8
    places = sum(BEGIN + max(1, -(-int(n) // TILE)) for n in lens) * -(-group // columns)
    shares = 152 * (1 if dim * columns >= 2048 else 2)
    return places / shares / (8 // heads)


@pytest.mark.parametrize("heads,dim,group,page,rows", [
    (8, 64, 2, 16, 300), (8, 128, 1, 32, 300), (4, 128, 2, 8, 400)])
def test_tiles_without_tokens_between_others(dk, heads, dim, group, page, rows):  # noqa: F811
    """A tile that no page is in the cache for completes without a copy: its
    mask has to be published all the same, in a stage that held other tokens."""
    rng = np.random.default_rng(heads + dim)
    cache, host = fill(dk, rng, 40, page, heads, dim)
    table, lens = walk(rng, 40, page, rows, 1536, rows // 8)
    for t in range(rows):  # spans of one to three tiles, at any page
        for at in rng.choice(1536 // page, 4, replace=False):
            table[t, at:at + rng.integers(1, 4) * max(1, TILE // page)] = rng.choice([-1, 40, 2 ** 30])
    table[rows // 2] = -1
    q, values = query(rng, rows, heads * group, dim, "f16")
    assert tiles_of_a_group(heads, dim, group, lens) >= 2 * STAGES
    assert dk.kv4_attention_workspace_size(cache, rows, heads * group, table.shape[1]) > 0
    out, lse = check(dk, cache, host, q, values, "f16", table, lens)
    again = dk.kv4_attention(cache, q, i32(table), i32(lens))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert dk.dcp_topk_device_status() == 0


@pytest.mark.parametrize("heads,dim,group,page,rows,dtype", [
    (8, 64, 1, 16, 300, "bf16"), (8, 64, 9, 8, 300, "f16"), (8, 64, 17, 64, 160, "bf16"),
    (8, 128, 2, 16, 300, "bf16"), (8, 128, 17, 32, 160, "f16"), (8, 256, 1, 128, 160, "f16"),
    (4, 128, 8, 16, 400, "f16"), (4, 128, 19, 8, 200, "bf16"), (4, 256, 9, 64, 160, "bf16")])
def test_walks_of_many_tiles(dk, heads, dim, group, page, rows, dtype):  # noqa: F811
    """Shares of ten places and more, pieces that begin and end anywhere, rows of
    nothing, windows; the same with weights."""
    rng = np.random.default_rng(heads * dim + group)
    cache, host = fill(dk, rng, 64, page, heads, dim)
    table, lens = walk(rng, 64, page, rows, 1536, rows // 8)
    starts = np.where(rng.random(rows) < 0.3, rng.integers(0, 1536, rows), 0)
    q, values = query(rng, rows, heads * group, dim, dtype)
    assert tiles_of_a_group(heads, dim, group, np.maximum(lens - starts, 0)) * (8 // heads) >= 10
    assert dk.kv4_attention_workspace_size(cache, rows, heads * group, table.shape[1]) > 0
    out, lse = check(dk, cache, host, q, values, dtype, table, lens, starts=starts)
    again = dk.kv4_attention(cache, q, i32(table), i32(lens), starts=i32(starts))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    w = torch.zeros(rows, 1536, device="cuda")
    out2, lse2 = dk.kv4_attention(cache, q, i32(table), i32(lens), starts=i32(starts), weights=w)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # a row's weights sum to its query heads, each head's to 1 within the fp32
    # sums of 1536 tokens, and lie inside its window
    pos = torch.arange(1536, device="cuda")
    seen = (pos >= i32(starts)[:, None]) & (pos < i32(lens)[:, None])
    total = torch.where(seen.any(1), heads * group, 0).double()
    assert ((w.double().sum(1) - total).abs() <= total * 1e-5).all()
    assert not w[~seen].any() and (w >= 0).all()
    assert dk.dcp_topk_device_status() == 0

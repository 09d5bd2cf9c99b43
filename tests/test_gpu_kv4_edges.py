"""Edges of the 4-bit cache's operators on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")

from .test_gpu_kv4 import DEV, dk, i32  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["softcap", "scale"])
def test_a_scale_or_cap_that_is_not_finite_is_refused(dk, name):  # noqa: F811
    cache = dk.Kv4Cache.allocate(1, 4, 1, 64, DEV)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    for value in (float("inf"), -float("inf"), float("nan"), 1e39):  # the last: no float
        with pytest.raises(ValueError, match=name):
            dk.kv4_attention(cache, q, i32([[0]]), i32([1]), **{name: value})


@pytest.mark.parametrize("q_size,key,named", [
    (3e38, 0.0, dict(scale=1e6)),       # products of 0 with what is beyond fp32
    (1.0, 0.0, dict(softcap=1e-44)),
    (1.0, 3.0, dict(softcap=1e-44))])   # every score at the cap
def test_equal_scores_whose_multiplier_leaves_fp32(dk, q_size, key, named):  # noqa: F811
    cache = dk.Kv4Cache.allocate(4, 16, 1, 64, DEV)
    x = torch.ones(64, 1, 64, device=DEV)
    dk.kv4_append(cache, key * x, 3 * x, torch.arange(64, device=DEV))
    q = torch.full((1, 4, 64), q_size, device=DEV).bfloat16()
    out, lse = dk.kv4_attention(cache, q, i32([[0, 1, 2, 3]]), i32([50]), **named)
    assert (out == 3).all()  # the mean of equal values: 3 / 6 and 6 are exact
    assert (lse - math.log(50)).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("with_ids", [False, True])
@pytest.mark.parametrize("q_heads", [3, 4])
def test_weights_of_a_nan_head_stay_with_tokens_that_are_there(dk, q_heads, with_ids):  # noqa: F811
    cache = dk.Kv4Cache.allocate(4, 16, 1, 64, DEV)
    x = torch.ones(64, 1, 64, device=DEV)
    dk.kv4_append(cache, x, x, torch.arange(64, device=DEV))
    q = torch.ones(2, q_heads, 64, dtype=torch.bfloat16, device=DEV)
    q[0, 1, 7] = float("nan")
    w = torch.zeros(2, 60, device=DEV)
    table = i32([[0, -1, 2, 4], [3, 99, 1, 0]])  # positions 16..31 are holes, row 0's 48..63, too
    ids = i32([list(range(60)) + [-1] * 9] * 2) if with_ids else None
    dk.kv4_attention(cache, q, table, i32([60, 40]), ids=ids, starts=i32([4, 0]), weights=w)
    there = torch.tensor([4 <= p < 16 or 32 <= p < 48 for p in range(60)], device=DEV)
    assert torch.isnan(w[0, there]).all() and not w[0, ~there].any()
    assert (w[1, :16] > 0).all() and (w[1, 32:40] > 0).all()
    assert not w[1, 16:32].any() and not w[1, 40:].any()


def test_eviction_leaves_nothing_old_where_a_hole_was_kept(dk):  # noqa: F811
    """The pages that an eviction fills may hold another sequence's tokens."""
    cache = dk.Kv4Cache.allocate(8, 4, 2, 64, DEV)
    planes = cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales
    for i, plane in enumerate(planes):
        plane.fill_(17 + i)
        plane[6:] = 51 + i
    w = torch.arange(24, dtype=torch.float32, device=DEV).view(2, 12)
    kept, lens, _ = dk.kv4_evict(cache, i32([[0, -1, 2], [3, 4, 8]]), i32([12, 12]), w,
                                 i32([[6], [7]]), 4, sinks=1, recent=1)
    assert kept.tolist() == [[0, 9, 10, 11], [0, 9, 10, 11]]
    kept2, _, _ = dk.kv4_evict(cache, i32([[-1, 1, 2]]), i32([4]), w[:1], i32([[5]]), 4)
    assert kept2.tolist() == [[0, 1, 2, 3]]
    for i, plane in enumerate(planes):
        assert (plane[6] == 17 + i).all()
        assert (plane[7, 0] == 17 + i).all() and not plane[7, 1:].any()
        assert not plane[5].any() and (plane[:5] == 17 + i).all()


@pytest.mark.parametrize("with_ids", [False, True])
@pytest.mark.parametrize("heads,width", [(1, 5), (8, 5), (8, 3000)])
def test_rows_of_a_table_without_sequences_see_nothing(dk, heads, width, with_ids):  # noqa: F811
    """Every owner is outside an empty table, which has no address."""
    cache = dk.Kv4Cache.allocate(2, 16, heads, 64, DEV)
    table = torch.zeros(0, width, dtype=torch.int32, device=DEV)
    q = torch.ones(3, 2 * heads, 64, dtype=torch.bfloat16, device=DEV)
    ids = i32([list(range(40))] * 3) if with_ids else None
    out, lse = dk.kv4_attention(cache, q, table, i32([5, 40, 0]), owner=i32([0, -1, 7]), ids=ids)
    assert not out.any() and torch.isneginf(lse).all()

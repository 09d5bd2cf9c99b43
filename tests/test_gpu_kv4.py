"""The 4-bit key/value cache on the GPU against its definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import kv4_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dk():
    import sparse_attention_indexer_stable_gb300 as dk
    return dk


def normal(rng, *shape, spread=0.7):
    """Normal values whose channels differ in size."""
    return rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[-1]))


def fill(dk, rng, pages, page, heads, dim, units=(1.0, 1.0)):
    """A cache full of quantised normal values, and its planes on the host."""
    planes = []
    for u in units:
        codes, scales = ref.encode(normal(rng, pages, page, heads, dim) * u, u)
        planes.append((ref.pack(codes), scales.astype(np.uint8)))
    host = (planes[0][0], planes[1][0], planes[0][1], planes[1][1])
    cache = dk.Kv4Cache(*[torch.from_numpy(np.ascontiguousarray(p)).to(DEV) for p in host],
                        k_unit=units[0], v_unit=units[1])
    return cache, host


def i32(x):
    return None if x is None else torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def query(rng, rows, heads, dim, dtype, strided=False, size=2.0):
    """Queries as a user has them: contiguous, or a slice of a wider buffer at
    an odd offset.  Returns (tensor, its values)."""
    x = torch.from_numpy(normal(rng, rows, heads, dim, spread=0.2) * size).to(TYPES[dtype]).to(DEV)
    if strided:
        flat = torch.zeros(rows * (heads + 2) * (dim + 3) + 1, dtype=x.dtype, device=DEV)[1:]
        view = flat.view(rows, heads + 2, dim + 3)[:, 1:1 + heads, 1:1 + dim]
        view.copy_(x)
        x = view
    return x, x.double().cpu().numpy()


def half_ulp(dtype):
    """The type's unit roundoff: 8 and 11 significant bits."""
    return {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]


def check(dk, cache, host, q, values, dtype, table, lens, *, units=(1.0, 1.0), **kw):
    """One call against the definition; returns (out, lse)."""
    named = {k: kw.pop(k) for k in ("ids", "owner", "starts", "row_starts") if k in kw}
    out, lse = dk.kv4_attention(cache, q, i32(table), i32(lens),
                                **{k: i32(v) for k, v in named.items()}, **kw)
    max_len = kw.get("max_len", 0)
    cut = np.minimum(lens, max_len) if max_len else lens
    want, want_lse, _, tol, lse_tol, _ = ref.attention(
        host, values, np.asarray(table), cut, units=units, **named,
        scale=kw.get("scale"), softcap=kw.get("softcap", 0.0))
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(got[empty] == 0)
    ok = ~empty
    # the type's rounding, and fp16's smallest step
    tol = tol * (1 + 2.0 ** -8) + half_ulp(dtype) * np.abs(want) + 2.0 ** -25
    worst = np.max(np.abs(got - want) - tol)
    assert worst <= 0, worst
    assert np.all(np.abs(got_lse[ok] - want_lse[ok]) <= lse_tol[ok])
    return out, lse


def table_of(rng, sequences, width, pages):
    """Every sequence's pages, no page twice while they last."""
    order = rng.permutation(max(pages, 1))
    return np.resize(order, (sequences, width)).astype(np.int32)


# ------------------------------------------------------------ append, read
def store_inputs(rng, n, heads, dim, dtype):
    x = normal(rng, n, heads, dim)
    x[0, 0, :16] = 0.0                           # a block of zeros
    x[-1, -1, 16:32] = [0.25 * i for i in range(-8, 8)]
    x[-1, 0, :16] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 2) * 1.125  # ties
    x[-1, 0, 32:48] = 1e-5                       # a scale that rounds to 0
    x[0, -1, 48:64] = 30000.0                    # a scale beyond the largest
    return torch.from_numpy(x).to(TYPES[dtype]).to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,heads,dim,page,units", [
    (1, 1, 64, 1, (1.0, 1.0)), (3, 5, 128, 16, (0.25, 4.0)), (130, 2, 256, 2, (1.0, 0.5)),
    (67, 8, 64, 64, (1.0, 1.0))])
def test_append_writes_exact_codes_and_read_returns_them(dk, dtype, n, heads, dim, page, units):
    rng = np.random.default_rng(n * dim)
    k, v = store_inputs(rng, n, heads, dim, dtype), store_inputs(rng, n, heads, dim, dtype)
    pages = -(-n // page) + 1
    cache = dk.Kv4Cache.allocate(pages, page, heads, dim, DEV, *units)
    slots = rng.permutation(pages * page)[:n]
    dk.kv4_append(cache, k, v, torch.from_numpy(slots).to(DEV))
    for x, u, codes, scales in ((k, units[0], cache.k_codes, cache.k_scales),
                                (v, units[1], cache.v_codes, cache.v_scales)):
        want_c, want_s = ref.encode(x.double().cpu().numpy(), u)
        got_c = codes.flatten(0, 1).cpu().numpy()
        assert np.array_equal(scales.flatten(0, 1).cpu().numpy()[slots], want_s)
        # equal values: a zero may carry either sign
        want = ref.decode(ref.pack(want_c), want_s, u)
        assert np.array_equal(ref.decode(got_c[slots], want_s, u), want)
        rest = np.setdiff1d(np.arange(pages * page), slots)
        assert not got_c[rest].any()
    back = dk.kv4_read(cache, torch.from_numpy(slots).to(DEV), dtype=torch.float32)
    for got, codes, scales, u in ((back[0], cache.k_codes, cache.k_scales, units[0]),
                                  (back[1], cache.v_codes, cache.v_scales, units[1])):
        want = ref.decode(codes.flatten(0, 1).cpu().numpy()[slots],
                          scales.flatten(0, 1).cpu().numpy()[slots], u)
        assert np.array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("unit", [1.0, 2.0 ** -20, 2.0 ** 20])
def test_append_codes_of_every_significand(dk, dtype, unit):
    """Blocks over all scales and all 16-bit significands, midpoints of the grid
    and their neighbours among them: every code and scale exact."""
    rng = np.random.default_rng(31)
    n, dim = 4096, 256
    scale = ref.SCALES[rng.integers(24, 120, (n, 1, dim // 16, 1))]
    x = rng.uniform(-6, 6, (n, 1, dim // 16, 16))
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], x.shape) * rng.choice([-1, 1], x.shape)
    x = np.where(rng.random(x.shape) < 0.5, ties, x)
    x[..., 0] = 6.0  # the block's scale
    x = (x * scale * (unit if dtype == "bf16" else 1.0)).reshape(n, 1, dim)
    t = torch.from_numpy(x).to(TYPES[dtype])
    near = t.view(torch.int16) + torch.from_numpy(rng.integers(-1, 2, x.shape).astype(np.int16))
    t = torch.where(torch.from_numpy(rng.random(x.shape) < 0.3), near.view(t.dtype), t).to(DEV)
    u = unit if dtype == "bf16" else 1.0
    cache = dk.Kv4Cache.allocate(1, n, 1, dim, DEV, u, u)
    dk.kv4_append(cache, t, t, torch.arange(n, device=DEV))
    want_c, want_s = ref.encode(t.double().cpu().numpy(), u)
    assert np.array_equal(cache.k_scales[0].cpu().numpy(), want_s)
    want = ref.decode(ref.pack(want_c), want_s)
    got = ref.decode(cache.k_codes[0].cpu().numpy(), want_s)
    assert np.array_equal(got, want)
    assert torch.equal(cache.k_codes, cache.v_codes)


def test_append_takes_strided_and_unaligned_values(dk):
    rng = np.random.default_rng(5)
    n, heads, dim = 9, 3, 64
    x = store_inputs(rng, n, heads, dim, "bf16")
    flat = torch.zeros(n * heads * (dim + 5) + 1, dtype=x.dtype, device=DEV)[1:]
    odd = flat.view(n, heads, dim + 5)[:, :, 2:2 + dim]
    odd.copy_(x)
    turned = x.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    slots = torch.arange(n, device=DEV)
    caches = []
    for k, v in ((x, x), (odd, turned)):
        cache = dk.Kv4Cache.allocate(1, 16, heads, dim, DEV)
        dk.kv4_append(cache, k, v, slots)
        caches.append(cache)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name))


def test_append_skips_slots_outside_and_read_gives_zeros(dk):
    rng = np.random.default_rng(6)
    x = store_inputs(rng, 4, 2, 128, "f32")
    cache = dk.Kv4Cache.allocate(2, 4, 2, 128, DEV)
    slots = torch.tensor([-1, 8, 7, 1 << 40], device=DEV)
    dk.kv4_append(cache, x, x, slots)
    written = cache.k_scales.flatten(0, 1).flatten(1).any(1).nonzero().flatten().tolist()
    assert written == [7]
    k, v = dk.kv4_read(cache, slots)
    assert not k[[0, 1, 3]].any() and not v[[0, 1, 3]].any() and k[2].any()
    dk.kv4_append(cache, x[:0], x[:0], slots[:0])
    assert dk.kv4_read(cache, slots[:0])[0].shape == (0, 2, 128)


def test_append_of_nan_and_infinity(dk):
    x = torch.ones(1, 1, 64, device=DEV)
    x[0, 0, 0], x[0, 0, 16], x[0, 0, 17], x[0, 0, 32:48] = float("nan"), float("inf"), -float("inf"), float("nan")
    cache = dk.Kv4Cache.allocate(1, 1, 1, 64, DEV)
    dk.kv4_append(cache, x, x, torch.zeros(1, dtype=torch.int64, device=DEV))
    k = dk.kv4_read(cache, torch.zeros(1, dtype=torch.int64, device=DEV), dtype=torch.float32)[0]
    one = ref.SCALES[ref.nearest(np.array(1 / 6), ref.SCALES)]
    near = one * ref.MAGNITUDES[ref.nearest(np.array(1 / one), ref.MAGNITUDES)]
    k = k[0, 0].cpu().numpy()
    assert k[0] == 0 and np.all(k[1:16] == np.float32(near))
    assert k[16] == 6 * 448 and k[17] == -6 * 448 and np.all(k[18:32] == 0)
    assert np.all(k[32:48] == 0)


# --------------------------------------------------------------- attention
EDGES = [0, 1, 2, 15, 16, 17, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,heads,group,page", [
    (64, 3, 1, 16), (64, 1, 12, 4), (128, 2, 8, 64), (128, 1, 3, 1), (128, 2, 16, 32),
    (128, 1, 21, 16), (256, 2, 4, 16), (256, 1, 9, 128)])
def test_dense_attention_at_edge_lengths(dk, dtype, dim, heads, group, page):
    rng = np.random.default_rng(dim + heads * group)
    width = -(-max(EDGES) // page)
    cache, host = fill(dk, rng, len(EDGES) * width, page, heads, dim)
    table = table_of(rng, len(EDGES), width, cache.num_pages)
    q, values = query(rng, len(EDGES), heads * group, dim, dtype)
    check(dk, cache, host, q, values, dtype, table, np.array(EDGES))


@pytest.mark.parametrize("width", [80, 1200])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 2), (256, 2), (64, 20), (128, 17), (256, 9)])
@pytest.mark.parametrize("lens", [[5000], [1, 4999, 777], [0, 0]])
def test_few_long_rows_are_split_and_joined(dk, dim, group, lens, width):
    """Cut into slices of a cluster (the narrow table) or into even shares
    (the wide one, as if rows could be long), the pieces joined."""
    rng = np.random.default_rng(sum(lens) + dim)
    cache, host = fill(dk, rng, 100, 64, 1, dim)
    table = table_of(rng, len(lens), width, 100)
    q, values = query(rng, len(lens), group, dim, "bf16")
    need = dk.kv4_attention_workspace_size(cache, len(lens), group, width)
    assert (need > 0) == (width == 1200)  # only shares need a workspace
    out, lse = check(dk, cache, host, q, values, "bf16", table, np.array(lens))
    again = dk.kv4_attention(cache, q, i32(table), i32(lens))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    # a bound of the lengths changes the split, and cuts longer rows
    check(dk, cache, host, q, values, "bf16", table, np.array(lens), max_len=max(1, max(lens)))
    check(dk, cache, host, q, values, "bf16", table, np.array(lens), max_len=300)


def test_even_shares_over_many_rows_of_all_lengths(dk):
    """Shares that begin and end inside rows, rows of no tokens between them,
    several heads and head tiles, for a range and for ids."""
    rng = np.random.default_rng(22)
    cache, host = fill(dk, rng, 60, 64, 2, 64)
    rows = 310
    lens = rng.integers(0, 700, rows)
    lens[rng.random(rows) < 0.3] = 0
    lens[[0, 1, 150, 309]] = [0, 3000, 3840, 0]
    table = table_of(rng, rows, 300, 60)
    q, values = query(rng, rows, 2 * 18, 64, "f16")
    assert dk.kv4_attention_workspace_size(cache, rows, 36, 300) > 0
    check(dk, cache, host, q, values, "f16", table, lens)
    few = slice(145, 155)
    ids = rng.permuted(np.tile(np.arange(19200), (10, 1)), axis=1)
    assert dk.kv4_attention_workspace_size(cache, 10, 36, 300, num_ids=19200) > 0
    check(dk, cache, host, q[few], values[few], "f16", table[few], lens[few], ids=ids)


@pytest.mark.parametrize("with_ids", [False, True])
@pytest.mark.parametrize("heads,dim,group", [
    (8, 128, 2), (7, 128, 1), (13, 128, 1), (5, 128, 3), (2, 128, 12), (8, 64, 2), (6, 64, 1),
    (12, 64, 1), (4, 64, 9), (7, 64, 1), (4, 256, 2), (3, 256, 1)])
def test_even_shares_of_all_head_counts(dk, heads, dim, group, with_ids):
    """Heads walked together in teams, part teams, teams with nobody, scale rows
    that are no whole 16-byte pieces; holes, windows, a row of nothing."""
    rng = np.random.default_rng(heads * dim + group)
    page, width = 16, 3000  # as if rows could be long: shares
    cache, host = fill(dk, rng, 48, page, heads, dim)
    rows = 4
    table = table_of(rng, rows, width, 48)
    table[0, 3], table[2, :2] = -1, [48, 2 ** 30]
    lens, starts = np.array([700, 0, 300, 33]), np.array([5, 0, 130, 32])
    ids = None
    if with_ids:
        ids = rng.integers(0, 720, (rows, 90000))
        ids[:, ::3] = -1
        ids[3] = -1
        ids[:, 200:] = -1
    q, values = query(rng, rows, heads * group, dim, "f16")
    assert dk.kv4_attention_workspace_size(cache, rows, heads * group, width,
                                           num_ids=90000 if with_ids else None) > 0
    out, lse = check(dk, cache, host, q, values, "f16", table, lens, starts=starts, ids=ids)
    w = torch.zeros(rows, 720, device=DEV)
    out2, lse2 = dk.kv4_attention(cache, q, i32(table), i32(lens), starts=i32(starts),
                                  ids=i32(ids), weights=w)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    _, _, want, _, _, tol = ref.attention(host, values, table, lens, ids=ids, starts=starts,
                                          positions=720)
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= tol + 2.0 ** -23 * want)


@pytest.mark.parametrize("heads,dim,group,page", [
    (8, 128, 8, 64), (8, 128, 1, 8), (8, 128, 20, 16), (8, 64, 3, 16), (8, 64, 9, 32),
    (8, 256, 2, 8), (4, 128, 8, 128), (4, 128, 12, 16), (4, 256, 5, 32), (8, 128, 2, 4)])
def test_even_shares_by_runs_of_a_page(dk, heads, dim, group, page):
    """All heads of 8 tokens copied at once: windows that begin anywhere, NaN
    scales in every slot that no row sees, holes, lengths that are no row's."""
    rng = np.random.default_rng(heads + dim + group + page)
    rows, pages, width = 7, 640 // page * 7, 48000 // page
    cache, host = fill(dk, rng, pages, page, heads, dim)
    table = np.full((rows, width), -1)
    table[:, :640 // page] = rng.permutation(pages).reshape(rows, -1)
    hole = 320 // page
    table[0, hole], table[2, hole:hole + 2] = -1, [pages, 2 ** 30]
    lens, starts = np.array([640, 0, 637, 33, 1, 500, -3]), np.array([5, 0, 131, 32, 0, 483, 0])
    pos = np.arange(width * page)
    for t in range(rows):  # poison what the row does not see
        unseen = np.flatnonzero((pos[:640] < starts[t]) | (pos[:640] >= lens[t]))
        slots = table[t, unseen // page] * page + unseen % page
        slots = slots[(slots >= 0) & (slots < pages * page)]
        for name in ("k_scales", "v_scales", "k_codes", "v_codes"):
            getattr(cache, name).view(pages * page, heads, -1)[torch.from_numpy(slots).to(DEV)] = 255
    q, values = query(rng, rows, heads * group, dim, "bf16")
    assert dk.kv4_attention_workspace_size(cache, rows, heads * group, width) > 0
    for softcap in (0.0, 20.0):
        out, lse = check(dk, cache, host, q, values, "bf16", table, lens, starts=starts,
                         softcap=softcap)
    w = torch.zeros(rows, 640, device=DEV)
    out2, lse2 = dk.kv4_attention(cache, q, i32(table), i32(lens), starts=i32(starts), weights=w,
                                  softcap=20.0)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    _, _, want, _, _, tol = ref.attention(host, values, table, np.maximum(lens, 0), starts=starts,
                                          positions=640, softcap=20.0)
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= tol + 2.0 ** -23 * want)
    assert dk.dcp_topk_device_status() == 0


def test_starts_negative_lengths_and_lengths_beyond_the_table(dk):
    rng = np.random.default_rng(7)
    cache, host = fill(dk, rng, 40, 16, 2, 128)
    table = table_of(rng, 7, 5, 40)
    lens = np.array([80, 200, -3, 50, 50, 50, 2 ** 31 - 1])
    starts = np.array([79, 3, 0, 50, 60, -7, 2 ** 31 - 1])
    q, values = query(rng, 7, 8, 128, "bf16")
    check(dk, cache, host, q, values, "bf16", table, lens, starts=starts)


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("softcap,scale,units", [
    (0.0, 0.31, (1.0, 1.0)), (3.0, None, (1.0, 1.0)), (30.0, 1.5, (0.125, 16.0)),
    (0.0, -0.1, (4.0, 2.0 ** -10))])
def test_scale_cap_units_and_strides(dk, strided, softcap, scale, units):
    rng = np.random.default_rng(11)
    cache, host = fill(dk, rng, 30, 16, 2, 128, units)
    table = table_of(rng, 3, 10, 30)
    q, values = query(rng, 3, 8, 128, "f16", strided=strided)
    check(dk, cache, host, q, values, "f16", table, np.array([150, 33, 4]), units=units,
          softcap=softcap, scale=scale)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-6, 1e4, 1e28])
def test_queries_of_any_size(dk, size):
    """bf16 queries far outside fp16's range: rows are scaled exactly."""
    rng = np.random.default_rng(12)
    cache, host = fill(dk, rng, 10, 16, 1, 64)
    table = table_of(rng, 2, 5, 10)
    q, values = query(rng, 2, 3, 64, "bf16", size=size)
    scale = float(np.float32(0.5 / size)) if size > 1e-30 else 1e30
    check(dk, cache, host, q, values, "bf16", table, np.array([80, 9]), scale=scale)


def test_holes_and_garbage_are_never_read_into_a_result(dk):
    """Pages outside the cache are absent, whole rows of them empty; unwritten
    slots that hold NaN scales reach no result."""
    rng = np.random.default_rng(13)
    cache, host = fill(dk, rng, 12, 16, 2, 128)
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    table[0, 1], table[1, :] = -1, [12, 2 ** 31 - 1, -5, 99]
    lens = np.array([50, 64, 33])
    for plane, value in ((2, 0x7F), (3, 0x7F), (0, 0xFF), (1, 0xFF)):
        host[plane][11, :] = value        # beyond row 2's end
        host[plane][10, 1:] = value
    for name, plane in zip(("k_codes", "v_codes", "k_scales", "v_scales"), host):
        getattr(cache, name).copy_(torch.from_numpy(plane))
    q, values = query(rng, 3, 4, 128, "bf16")
    check(dk, cache, host, q, values, "bf16", table, lens)


def test_infinite_and_nan_queries_spread_no_further_than_their_head(dk):
    rng = np.random.default_rng(14)
    cache, host = fill(dk, rng, 10, 16, 1, 64)
    table = table_of(rng, 1, 10, 10)
    q, values = query(rng, 1, 4, 64, "f16")
    clean, lse = dk.kv4_attention(cache, q, i32(table), i32([150]))
    q[0, 1, 5], q[0, 2, 7] = float("nan"), float("inf")
    out, lse2 = dk.kv4_attention(cache, q, i32(table), i32([150]))
    for h in (0, 3):
        assert torch.equal(out[0, h], clean[0, h]) and lse2[0, h] == lse[0, h]
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse2[0, 1])
    assert torch.isnan(out[0, 2]).all()


@pytest.mark.parametrize("owned", [False, True])
@pytest.mark.parametrize("dim,heads,group,num_ids", [
    (128, 2, 8, 300), (64, 1, 1, 1), (256, 1, 4, 17), (128, 1, 16, 2048), (128, 4, 2, 0)])
def test_selected_ids(dk, owned, dim, heads, group, num_ids):
    """Padding, ids outside the row's range, repeated ids, row starts."""
    rng = np.random.default_rng(num_ids + dim)
    cache, host = fill(dk, rng, 64, 16, heads, dim)
    rows = 5
    table = table_of(rng, 2 if owned else rows, 30, 64)
    owner = np.array([0, 1, 1, 0, 1]) if owned else None
    lens = np.array([480, 200, 31, 1, 0])
    row_starts = np.array([0, 1000, -5, 7, 3])
    ids = rng.integers(0, 500, (rows, num_ids)) + row_starts[:, None]
    ids[rng.random(ids.shape) < 0.2] = -1
    q, values = query(rng, rows, heads * group, dim, "bf16")
    check(dk, cache, host, q, values, "bf16", table, lens, ids=ids, owner=owner,
          row_starts=row_starts, starts=np.array([0, 20, 0, 0, 0]))


@pytest.mark.parametrize("heads,dim,group,rows,num_ids", [
    (8, 128, 2, 75, 300), (2, 128, 7, 160, 623), (2, 128, 12, 100, 511), (2, 128, 40, 50, 330),
    (4, 64, 3, 120, 821), (8, 64, 9, 50, 512), (8, 128, 1, 9, 2048), (4, 64, 1, 24, 2500),
    (6, 128, 3, 40, 1000)])
def test_selected_ids_of_many_short_rows(dk, heads, dim, group, rows, num_ids):
    """Neighbouring heads' warps copy together: rows of one to many tiles of 32
    ids, rows of nothing, windows, holes, padding, head tiles; whole rows to a
    CTA and rows split over a cluster."""
    rng = np.random.default_rng(heads * dim + group)
    cache, host = fill(dk, rng, 100, 16, heads, dim)
    table = table_of(rng, rows, 60, 100)
    table[0, 3], table[2, :2] = -1, [100, 2 ** 30]
    lens = rng.integers(1, 960, rows)
    lens[[1, 4]] = [0, 1]
    starts = np.where(rng.random(rows) < 0.5, lens // 3, 0)
    ids = rng.integers(0, 960, (rows, num_ids))
    ids[:, ::5] = -1
    ids[3] = -1
    ids[5, 33:] = -1
    ids[6:8, :num_ids // 2] = -1
    q, values = query(rng, rows, heads * group, dim, "bf16")
    # slices: no workspace; enough of them for teams
    assert dk.kv4_attention_workspace_size(cache, rows, heads * group, 60, num_ids=num_ids) == 0
    width = 8 if group <= 8 else 16
    assert rows * heads * -(-group // width) * -(-num_ids // 32) * dim >= 20 * 128 * 152
    out, lse = check(dk, cache, host, q, values, "bf16", table, lens, starts=starts, ids=ids)
    w = torch.zeros(rows, 960, device=DEV)
    out2, lse2 = dk.kv4_attention(cache, q, i32(table), i32(lens), starts=i32(starts),
                                  ids=i32(ids), weights=w)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    _, _, want, _, _, tol = ref.attention(host, values, table, lens, ids=ids, starts=starts,
                                          positions=960)
    assert np.all(np.abs(w.double().cpu().numpy() - want) <= tol + 2.0 ** -23 * want)


def test_ids_and_row_starts_at_the_ends_of_int32(dk):
    rng = np.random.default_rng(15)
    cache, host = fill(dk, rng, 8, 16, 1, 64)
    table = table_of(rng, 3, 8, 8)
    big = 2 ** 31 - 1
    ids = np.array([[big, big - 1, 0], [0, big, 3], [big, 5, -big - 1]])
    q, values = query(rng, 3, 2, 64, "f16")
    check(dk, cache, host, q, values, "f16", table, np.array([100, 100, 100]), ids=ids,
          row_starts=np.array([big - 9, -big - 1, -big]))


def test_owner_outside_the_table_sees_nothing(dk):
    rng = np.random.default_rng(16)
    cache, host = fill(dk, rng, 8, 16, 1, 64)
    table = table_of(rng, 2, 4, 8)
    q, values = query(rng, 4, 2, 64, "f16")
    check(dk, cache, host, q, values, "f16", table, np.array([60] * 4), owner=[1, 2, -1, 0])


def test_ids_select_the_same_as_the_range(dk):
    """All positions as ids, in the range's order: the same slices, the same bits."""
    rng = np.random.default_rng(17)
    cache, _ = fill(dk, rng, 64, 16, 2, 128)
    table = table_of(rng, 1, 64, 64)
    q, _ = query(rng, 1, 16, 128, "bf16")
    ids = np.arange(1024)[None]
    a = dk.kv4_attention(cache, q, i32(table), i32([1024]))
    b = dk.kv4_attention(cache, q, i32(table), i32([1024]), ids=i32(ids))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("with_ids", [False, True])
@pytest.mark.parametrize("dim,heads,group,lens", [
    (128, 2, 8, [300, 1, 0, 77]), (64, 3, 1, [40]), (256, 1, 11, [2500, 16])])
def test_weights_accumulate(dk, with_ids, dim, heads, group, lens):
    rng = np.random.default_rng(sum(lens))
    cache, host = fill(dk, rng, 200, 16, heads, dim)
    rows, width = len(lens), 160
    table = table_of(rng, rows, width, 200)
    table[0, 1] = -1
    q, values = query(rng, rows, heads * group, dim, "bf16")
    starts = np.array([n // 5 for n in lens])
    ids = None
    if with_ids:
        ids = np.stack([rng.permutation(2600)[:900] for _ in lens])
        ids[:, ::7] = -1
    positions = max(lens) - 10 if max(lens) > 100 else max(lens)  # narrower than a row
    base = torch.rand(rows, positions + 3, device=DEV)[:, :positions]
    before = base.clone()
    out, lse = dk.kv4_attention(cache, q, i32(table), i32(lens), ids=i32(ids), starts=i32(starts),
                                weights=base)
    plain, plain_lse = dk.kv4_attention(cache, q, i32(table), i32(lens), ids=i32(ids),
                                        starts=i32(starts))
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)
    _, _, want, _, _, tol = ref.attention(host, values, table, lens, ids=ids, starts=starts,
                                          positions=positions)
    got = base.double().cpu().numpy()
    old = before.double().cpu().numpy()
    # the addition to the old weight rounds once more
    assert np.all(np.abs(got - old - want) <= tol + 2.0 ** -23 * (old + want))
    assert np.array_equal(got[want == 0], old[want == 0])


def test_attention_on_another_stream_and_in_a_graph(dk):
    rng = np.random.default_rng(18)
    cache, host = fill(dk, rng, 100, 64, 2, 128)
    table = i32(table_of(rng, 2, 50, 100))
    q, values = query(rng, 2, 16, 128, "bf16")
    lens = i32([3000, 1700])
    want = dk.kv4_attention(cache, q, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dk.kv4_attention(cache, q, table, lens, stream=side)
    raw = dk.kv4_attention(cache, q, table, lens, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(raw[1], want[1])
    w = torch.zeros(2, 3200, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = dk.kv4_attention(cache, q, table, lens, weights=w)
    lens.copy_(i32([5, 1700]))
    graph.replay()
    torch.cuda.synchronize()
    fresh = dk.kv4_attention(cache, q, table, lens)
    assert torch.equal(captured[0], fresh[0]) and torch.equal(captured[1], fresh[1])
    sums = w.sum(1).cpu().numpy()
    assert np.all(np.abs(sums - 16) < 1e-3)  # every head's weights sum to 1


def test_given_outputs_and_workspace_are_used(dk):
    rng = np.random.default_rng(19)
    cache, host = fill(dk, rng, 100, 64, 1, 64)
    table = i32(table_of(rng, 1, 1000, 100))
    q, _ = query(rng, 1, 4, 64, "f16")
    need = dk.kv4_attention_workspace_size(cache, 1, 4, 1000)
    space = torch.empty(need, dtype=torch.uint8, device=DEV)
    out = torch.empty(1, 4, 64, dtype=torch.float16, device=DEV)
    lse = torch.empty(1, 4, device=DEV)
    got = dk.kv4_attention(cache, q, table, i32([6000]), out=out, lse=lse, workspace=space)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, dk.kv4_attention(cache, q, table, i32([6000]))[0])
    with pytest.raises(ValueError):
        dk.kv4_attention(cache, q, table, i32([6000]), workspace=space[:need - 1])


def test_no_rows_and_no_pages(dk):
    cache = dk.Kv4Cache.allocate(0, 16, 2, 64, DEV)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = dk.kv4_attention(cache, q, i32(np.zeros((0, 3))), i32([]))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    for width in (0, 3):
        out, lse = dk.kv4_attention(cache, q, i32(np.zeros((2, width))), i32([5, 40]))
        assert not out.any() and torch.isneginf(lse).all()


# ---------------------------------------------------------------- eviction
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([100, 64, 65, 0, 1], 64, 4, 16), ([5000, 4999, 31], 32, 0, 0), ([300, 40], 40, 40, 0),
    ([300, 41], 40, 0, 40), ([20000, 9000], 1000, 7, 33), ([70000], 300, 0, 1), ([9], 1, 0, 0),
    ([150000, 140001], 2000, 0, 100)])
@pytest.mark.parametrize("kind", ["ties", "zeros", "spread", "odd"])
def test_eviction_keeps_the_heaviest_in_order(dk, lens, budget, sinks, recent, kind):
    rng = np.random.default_rng(sum(lens) + budget)
    heads, dim, page = (1, 64, 16) if max(lens) > 10000 else (3, 128, 16)
    width = -(-max(lens) // page)
    per = -(-budget // page)
    B = len(lens)
    pages = B * (width + per)
    cache = dk.Kv4Cache.allocate(pages, page, heads, dim, DEV)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        t = getattr(cache, name)
        t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape), dtype=np.uint8)))
    order = rng.permutation(pages).astype(np.int32)
    table, out_table = order[:B * width].reshape(B, -1), order[B * width:].reshape(B, -1)
    w = {"ties": rng.integers(0, 4, (B, max(lens))) / 4, "zeros": np.zeros((B, max(lens))),
         "spread": np.exp(4 * rng.standard_normal((B, max(lens)))),
         "odd": rng.choice([0.0, -0.0, 1e-40, -1.0, np.inf, -np.inf, np.nan, 3.0],
                           (B, max(lens)))}[kind].astype(np.float32)
    before = {n: getattr(cache, n).flatten(0, 1).cpu().numpy()
              for n in ("k_codes", "v_codes", "k_scales", "v_scales")}
    kept, new_lens, new_w = dk.kv4_evict(cache, i32(table), i32(lens),
                                         torch.from_numpy(w).to(DEV), i32(out_table), budget,
                                         sinks=sinks, recent=recent)
    kept, new_w = kept.cpu().numpy(), new_w.cpu().numpy()
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    after = {n: getattr(cache, n).flatten(0, 1).cpu().numpy() for n in before}
    for b, n in enumerate(lens):
        want = ref.evict(n, w[b], budget, sinks, recent)
        assert np.array_equal(kept[b, :len(want)], want)
        assert np.all(kept[b, len(want):] == -1) and np.all(new_w[b, len(want):] == 0)
        assert np.array_equal(new_w[b, :len(want)], w[b, want], equal_nan=True)
        src = table[b, want // page] * page + want % page
        j = np.arange(len(want))
        dst = out_table[b, j // page] * page + j % page
        for name in before:
            assert np.array_equal(after[name][dst], before[name][src])
            before[name][dst] = before[name][src]
    for name in before:  # nothing else changed
        assert np.array_equal(after[name], before[name])


def test_eviction_with_holes_and_short_tables(dk):
    """Lengths beyond the weights or the table are cut; tokens on holes are
    kept by the rule but have nothing to copy."""
    cache = dk.Kv4Cache.allocate(6, 4, 1, 64, DEV)
    cache.k_codes.fill_(7)
    table, out = i32([[0, -1, 2], [3, 99, 4]]), i32([[5], [6]])
    w = torch.arange(20, dtype=torch.float32, device=DEV).view(2, 10)
    cache.k_codes[5] = 0
    kept, lens, _ = dk.kv4_evict(cache, table, i32([500, -4]), w, out, 4, sinks=1, recent=1)
    assert kept.tolist() == [[0, 7, 8, 9], [-1] * 4] and lens.tolist() == [4, 0]
    assert (cache.k_codes[5, [0, 2, 3]] == 7).all() and not cache.k_codes[5, 1].any()


def test_attention_after_eviction_is_attention_over_the_kept(dk):
    """Accumulate, evict, attend: the evicted cache answers as the kept ids do."""
    rng = np.random.default_rng(21)
    cache, host = fill(dk, rng, 60, 16, 2, 128)
    table, out_table = i32(np.arange(40).reshape(2, 20)), i32(np.arange(40, 60).reshape(2, 10))
    lens = i32([320, 200])
    q, _ = query(rng, 2, 8, 128, "bf16")
    w = torch.zeros(2, 320, device=DEV)
    dk.kv4_attention(cache, q, table, lens, weights=w)
    kept, new_lens, new_w = dk.kv4_evict(cache, table, lens, w, out_table, 128, sinks=4, recent=16)
    a = dk.kv4_attention(cache, q, out_table, new_lens, max_len=128)
    b = dk.kv4_attention(cache, q, table, lens, ids=kept)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (new_w.sum(1) >= w.sum(1) * 128 / 320).all()


# ---------------------------------------------------------------- refusals
def test_the_cache_refuses_planes_that_do_not_fit(dk):
    def planes(pages=2, page=4, heads=2, dim=64, device=DEV):
        return [torch.zeros(pages, page, heads, w, dtype=torch.uint8, device=device)
                for w in (dim // 2, dim // 2, dim // 16, dim // 16)]

    dk.Kv4Cache(*planes())
    for bad in (dict(page=3), dict(dim=32), dict(dim=192)):
        with pytest.raises(dk.DcpError) as e:
            dk.Kv4Cache(*planes(**bad))
        assert e.value.status == dk.DCP_ERR_UNSUPPORTED
    for unit in (0.0, 3.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(dk.DcpError) as e:
            dk.Kv4Cache(*planes(), k_unit=unit)
        assert e.value.status == dk.DCP_ERR_INVALID
    with pytest.raises(ValueError):
        dk.Kv4Cache(*planes(device="cpu"))
    p = planes()
    with pytest.raises(ValueError):
        dk.Kv4Cache(p[0], p[1], p[0], p[3])
    with pytest.raises(TypeError):
        dk.Kv4Cache(p[0].int(), *p[1:])
    with pytest.raises(ValueError):
        dk.Kv4Cache(p[0].transpose(0, 1), *p[1:])
    flat = torch.zeros(2 * 4 * 2 * 32 + 8, dtype=torch.uint8, device=DEV)[8:]
    with pytest.raises(dk.DcpError):  # not 16-byte aligned
        dk.Kv4Cache(flat.view(2, 4, 2, 32), *p[1:])


def test_attention_refuses_arguments_that_do_not_fit(dk):
    cache = dk.Kv4Cache.allocate(4, 4, 2, 64, DEV)
    good = dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV),
                table=i32(np.zeros((2, 2))), lens=i32([1, 2]))
    dk.kv4_attention(cache, **good)
    q = good["q"]
    bad = [
        (TypeError, dict(q=q.float())), (TypeError, dict(q=q.int())), (ValueError, dict(q=q.cpu())),
        (ValueError, dict(q=q[:, :3])), (ValueError, dict(q=q[..., :32])),
        (ValueError, dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))),
        (TypeError, dict(table=good["table"].long())), (ValueError, dict(table=good["table"][:1])),
        (ValueError, dict(table=good["table"][0])), (ValueError, dict(lens=i32([1]))),
        (TypeError, dict(lens=torch.zeros(2, device=DEV))), (ValueError, dict(starts=i32([0]))),
        (TypeError, dict(ids=torch.zeros(2, 3, dtype=torch.int64, device=DEV))),
        (ValueError, dict(ids=i32(np.zeros((1, 3))))), (ValueError, dict(owner=i32([0, 0, 0]))),
        (ValueError, dict(owner=i32([0, 0]), weights=torch.zeros(2, 8, device=DEV))),
        (ValueError, dict(weights=torch.zeros(1, 8, device=DEV))),
        (ValueError, dict(weights=torch.zeros(1, 8, device=DEV).expand(2, 8))),
        (ValueError, dict(softcap=-1.0)), (ValueError, dict(softcap=float("nan"))),
        (ValueError, dict(out=torch.zeros(2, 4, 32, dtype=torch.bfloat16, device=DEV))),
        (TypeError, dict(out=torch.zeros(2, 4, 64, device=DEV))),
        (dk.DcpError, dict(max_len=-1)),
    ]
    for error, change in bad:
        with pytest.raises(error):
            dk.kv4_attention(cache, **{**good, **change})
    with pytest.raises(TypeError):
        dk.kv4_attention(None, **good)


def test_store_and_eviction_refuse_arguments_that_do_not_fit(dk):
    cache = dk.Kv4Cache.allocate(4, 4, 2, 64, DEV)
    k = torch.zeros(3, 2, 64, device=DEV)
    slots = torch.arange(3, device=DEV)
    for error, args in ((TypeError, (k.double(), k, slots)), (ValueError, (k, k.half(), slots)),
                        (ValueError, (k[:2], k, slots)), (ValueError, (k, k, slots[:2])),
                        (TypeError, (k, k, slots.int())), (ValueError, (k[:, :1], k[:, :1], slots))):
        with pytest.raises(error):
            dk.kv4_append(cache, *args)
    with pytest.raises(TypeError):
        dk.kv4_read(cache, slots.int())
    with pytest.raises(TypeError):
        dk.kv4_read(cache, slots, dtype=torch.float64)
    good = dict(table=i32([[0, 1]]), lens=i32([8]), weights=torch.zeros(1, 8, device=DEV),
                out_table=i32([[2]]), budget=4)
    dk.kv4_evict(cache, **good)
    for error, change in ((ValueError, dict(budget=0)), (ValueError, dict(budget=5)),
                          (ValueError, dict(sinks=3, recent=2)), (ValueError, dict(sinks=-1)),
                          (TypeError, dict(weights=torch.zeros(1, 8, device=DEV).double())),
                          (ValueError, dict(weights=torch.zeros(2, 8, device=DEV))),
                          (ValueError, dict(lens=i32([8, 8]))),
                          (TypeError, dict(out_table=torch.zeros(1, 1, device=DEV)))):
        with pytest.raises(error):
            dk.kv4_evict(cache, **{**good, **change})

"""A batch's bookkeeping and rotary positions on the GPU against their definitions."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import prompt_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half a step, relative


@pytest.fixture(scope="module")
def dk():
    import sparse_attention_indexer_stable_gb300 as dk
    return dk


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), device=DEV).int()


# ------------------------------------------------------------------ extend
def batch(rng, B, page, longest, most, width=None, spare=None, pages_off=0):
    """(table, lens, counts, free, num_pages) of B sequences on the host."""
    lens = rng.integers(0, longest + 1, B)
    counts = rng.integers(0, most + 1, B)
    held = -(-lens // page)
    width = int(max(1, (-(-(lens + counts) // page)).max(initial=0))) if width is None else width
    need = int(held.sum()) + B * (most // page + 1)
    order = rng.permutation(need)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        n = min(int(held[b]), width)
        table[b, :n] = order[at:at + n]
        at += n
    free = order[at:] if spare is None else order[at:at + spare]
    return table, lens, counts, free, need - pages_off


def check_extend(dk, table, lens, counts, free, used, places, page, num_pages, pad=0, **kw):
    B, width = table.shape
    wide = torch.full((B, width + pad), 7, dtype=torch.int32, device=DEV)
    wide[:, :width] = i32(table)
    got_table = wide[:, :width]
    step = dk.kv4_extend(got_table, i32(lens), i32(counts), i32(free), i32([used]), places=places,
                         page_size=page, num_pages=num_pages, **kw)
    want = ref.extend(table, lens, counts, free, used, places, page, num_pages)
    for name, got, w in zip(step._fields, step, want):
        assert got.tolist() == w, name
    assert got_table.tolist() == want[7]
    assert (wide[:, width:] == 7).all()
    return step


@pytest.mark.parametrize("B,page,longest,most,extra", [
    (1, 1, 0, 1, 0), (1, 64, 100, 1, 0), (3, 16, 40, 50, 5), (7, 2, 9, 3, 1), (33, 64, 300, 200, 0),
    (1025, 16, 90, 1, 30), (2500, 4, 20, 9, 0), (16384, 8, 20, 2, 100), (5, 128, 1000, 3000, 100),
    (2, 65536, 70000, 9, 0)])
def test_extend_matches_the_definition(dk, B, page, longest, most, extra):
    rng = np.random.default_rng(B * page)
    table, lens, counts, free, pages = batch(rng, B, page, longest, most)
    check_extend(dk, table, lens, counts, free, 0, int(counts.sum()) + extra, page, pages, pad=3)


@pytest.mark.parametrize("change", ["short list", "used", "used past the list", "narrow table",
                                    "few places", "no places", "pages outside", "negative",
                                    "no free pages", "idle"])
def test_extend_at_its_edges(dk, change):
    rng = np.random.default_rng(11)
    kw = dict(spare=4) if change == "short list" else {}
    table, lens, counts, free, pages = batch(rng, 9, 8, 50, 40, **kw)
    used, places = 0, int(counts.sum()) + 2
    if change == "used":
        used = 3
    if change == "used past the list":
        used = len(free) + 5
    if change == "narrow table":
        table = table[:, :5]
    if change == "few places":
        places = int(counts.sum()) // 2
    if change == "no places":
        places = 0
    if change == "pages outside":  # entries of the list that the cache does not have, and holes
        pages -= 20
        table[2, 0] = -5
    if change == "negative":
        lens[1], counts[2], used = -4, -7, -1
    if change == "no free pages":
        free = free[:0]
    if change == "idle":
        counts[:] = 0
    check_extend(dk, table, lens, counts, free, used, places, 8, pages)


def test_extend_without_sequences(dk):
    step = dk.kv4_extend(torch.empty((0, 4), dtype=torch.int32, device=DEV), i32([]), i32([]),
                         i32([1, 2]), i32([1]), places=3, page_size=16, num_pages=4)
    assert [x.tolist() for x in step] == [[-1] * 3, [0] * 3, [-1] * 3, [0] * 3, [0], [], [1]]


def test_extend_lengths_stop_at_the_largest(dk):
    top = 2 ** 31 - 1
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    step = dk.kv4_extend(table, i32([top - 1, 3]), i32([top, 2]), i32([1]), i32([top]), places=4,
                         page_size=16, num_pages=4)
    assert step.slots.tolist() == [-1] * 4 and step.owner.tolist() == [0] * 4
    assert step.positions.tolist() == [top - 1, top, top, top]
    assert step.row_lens.tolist() == [top] * 4
    assert step.lens.tolist() == [top, 3] and step.used.tolist() == [top]


def test_extend_in_place_through_a_graph(dk):
    """Replays advance the lengths, the list and the table by a token each."""
    rng = np.random.default_rng(5)
    B, page = 6, 4
    table, lens, _, free, pages = batch(rng, B, page, 9, 30, width=12)
    t, n, u = i32(table), i32(lens), i32([0])
    step = dk.Kv4Step(torch.empty(8, dtype=torch.int64, device=DEV), *[
        torch.empty(8, dtype=torch.int32, device=DEV) for _ in range(3)],
        torch.empty(B + 1, dtype=torch.int32, device=DEV), n, u)
    counts = i32([1] * B)
    args = dict(places=8, page_size=page, num_pages=pages, out=step)
    f = i32(free)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = dk.kv4_extend(t, n, counts, f, u, **args)
    assert all(a is b for a, b in zip(got, step))
    torch.cuda.current_stream().wait_stream(side)
    host = (table, lens, [0])
    for _ in range(10):
        graph.replay()
        want = ref.extend(host[0], host[1], [1] * B, free, host[2][0], 8, page, pages)
        assert [x.tolist() for x in step] == list(want[:7]) and t.tolist() == want[7]
        host = (np.array(want[7]), want[5], want[6])


@pytest.mark.parametrize("B,most", [(40, 300), (1500, 9), (3, 30000)])
def test_extend_in_place_with_many_places(dk, B, most):
    """Lengths and the list's count in place, over all CTAs of a cluster."""
    rng = np.random.default_rng(B)
    table, lens, counts, free, pages = batch(rng, B, 16, 100, most)
    places = int(counts.sum()) + 50
    t, n, u = i32(table), i32(lens), i32([0])
    step = dk.Kv4Step(torch.empty(places, dtype=torch.int64, device=DEV), *[
        torch.empty(places, dtype=torch.int32, device=DEV) for _ in range(3)],
        torch.empty(B + 1, dtype=torch.int32, device=DEV), n, u)
    dk.kv4_extend(t, n, i32(counts), i32(free), u, places, 16, pages, out=step)
    want = ref.extend(table, lens, counts, free, 0, places, 16, pages)
    assert [x.tolist() for x in step] == list(want[:7]) and t.tolist() == want[7]


def test_extend_on_another_stream(dk):
    rng = np.random.default_rng(2)
    table, lens, counts, free, pages = batch(rng, 20, 16, 200, 100)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check_extend(dk, table, lens, counts, free, 0, int(counts.sum()), 16, pages)
    with torch.cuda.stream(s):
        check_extend(dk, table, lens, counts, free, 0, int(counts.sum()), 16, pages)
    s.synchronize()


@pytest.mark.parametrize("change", [
    dict(lens=torch.zeros(2, dtype=torch.int32)), dict(counts=torch.zeros(3, dtype=torch.int64)),
    dict(counts=torch.zeros(4, dtype=torch.int32)), dict(used=torch.zeros(2, dtype=torch.int32)),
    dict(free=torch.zeros(2, 2, dtype=torch.int32)), dict(table=torch.zeros(3, dtype=torch.int32)),
    dict(table=torch.zeros(1, 4, dtype=torch.int32).expand(3, 4)),
    dict(places=-1), dict(page_size=24), dict(num_pages=2 ** 40), dict(out=(1, 2)),
    dict(out=(None,) * 7)])
def test_extend_refusals(dk, change):
    a = dict(table=torch.zeros(3, 4, dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32),
             counts=torch.zeros(3, dtype=torch.int32), free=torch.zeros(2, dtype=torch.int32),
             used=torch.zeros(1, dtype=torch.int32), places=4, page_size=16, num_pages=9)
    a.update(change)
    host = "lens" in change  # left on the host
    a = {k: v.to(DEV) if isinstance(v, torch.Tensor) and not (host and k == "lens") else v
         for k, v in a.items()}
    if change.get("table") is not None and change["table"].stride(0) == 0:
        a["table"] = torch.zeros(1, 4, dtype=torch.int32, device=DEV).expand(3, 4)
    with pytest.raises((TypeError, ValueError, dk.DcpError)):
        dk.kv4_extend(**a)


# ------------------------------------------------------------------ rotary
def heads(rng, n, h, D, dtype, layout):
    """(tensor, values): contiguous, a slice of a wider buffer, or one whose
    rows and addresses allow no 16-byte accesses."""
    x = torch.from_numpy(rng.standard_normal((n, h, D)) * 3).to(TYPES[dtype]).to(DEV)
    if layout == "sliced":
        wide = torch.zeros(n, h + 4, D, dtype=x.dtype, device=DEV)
        wide[:, 2:2 + h] = x
        x = wide[:, 2:2 + h]
    if layout == "odd":
        flat = torch.zeros(n * (h + 1) * (D + 3) + 1, dtype=x.dtype, device=DEV)[1:]
        wide = flat.view(n, h + 1, D + 3)[:, 1:, 1:1 + D]
        wide.copy_(x)
        x = wide
    if layout == "heads first":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    return x, x.double().cpu().numpy()


def check_turned(rope, got, x, positions, dtype):
    want = ref.turned(x, positions, rope.frequencies, interleaved=rope.interleaved,
                      magnitude=rope.magnitude)
    size = np.abs(x).max(-1, keepdims=True)
    # cosine and sine of the fp32 angle within 4 half-steps, their product with
    # the magnitude, two products and a sum: 8 half-steps of both elements; the
    # rounding to the type, and fp16's smallest step
    tol = 16 * 2.0 ** -24 * size * abs(rope.magnitude) + STEP[dtype] * np.abs(want) * (
        1 + 2.0 ** -8) + 2.0 ** -25
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    R = 2 * len(rope.frequencies)
    assert np.array_equal(got.double().cpu().numpy()[..., R:], x[..., R:])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,D,R,layout", [
    (1, 1, 1, 64, 64, "plain"), (5, 8, 2, 128, 128, "sliced"), (3, 3, 1, 128, 64, "odd"),
    (33, 12, 12, 64, 32, "heads first"), (2, 4, 1, 256, 256, "plain"), (7, 2, 1, 96, 2, "plain"),
    (4, 5, 5, 80, 48, "sliced"), (1, 40, 8, 1024, 1024, "plain"), (9, 1, 1, 7, 6, "plain"),
    (2, 60, 10, 1023, 1022, "plain"), (3, 600, 1, 128, 128, "plain")])
def test_rotary_matches_the_definition(dk, dtype, interleaved, n, hq, hk, D, R, layout):
    rng = np.random.default_rng(n * D + R)
    rope = dk.Rotary(R, interleaved=interleaved)
    q, xq = heads(rng, n, hq, D, dtype, layout)
    k, xk = heads(rng, n, hk, D, dtype, layout)
    positions = rng.integers(-5, 200000, n)
    yq, yk = dk.rotary(rope, i32(positions), q, k)
    check_turned(rope, yq, xq, positions, dtype)
    check_turned(rope, yk, xk, positions, dtype)
    assert np.array_equal(q.double().cpu().numpy(), xq)  # the inputs are left alone


@pytest.mark.parametrize("kw", [
    dict(factor=8.0), dict(factor=8.0, original=4096), dict(base=1e6), dict(magnitude=-0.5),
    dict(factor=32.0, original=2048, slow=2.0, fast=8.0), dict(frequencies=[0.0, 3.0, -1e-3, 1e4])])
def test_rotary_far_positions_and_scalings(dk, kw):
    rng = np.random.default_rng(1)
    rope = dk.Rotary(8, **kw)
    positions = np.array([0, 1, -1, 4097, 10 ** 6 + 3, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31])
    q, x = heads(rng, len(positions), 3, 8, "f32", "plain")
    yq, none = dk.rotary(rope, i32(positions), q)
    assert none is None
    check_turned(rope, yq, x, positions, "f32")


def test_rotary_blends_by_turns(dk):
    """Frequencies of many turns are kept, of few divided, one between blended."""
    rope = dk.Rotary(128, factor=4.0, original=4096, slow=1.0, fast=32.0)
    plain = dk.Rotary(128)
    for f, g in zip(plain.frequencies, rope.frequencies):
        turns = 4096 * f / (2 * np.pi)
        want = f if turns >= 32 else f / 4 if turns <= 1 else None
        if want is not None:
            assert g == pytest.approx(want, rel=1e-15)
        else:
            assert f / 4 < g < f
    assert rope.magnitude == pytest.approx(0.1 * np.log(4.0) + 1)


@pytest.mark.parametrize("layout", ["plain", "sliced", "odd", "heads first"])
def test_rotary_in_place_and_back(dk, layout):
    rng = np.random.default_rng(3)
    rope = dk.Rotary(64, interleaved=True)
    q, xq = heads(rng, 17, 6, 128, "f32", layout)
    k, xk = heads(rng, 17, 2, 128, "f32", layout)
    positions = rng.integers(0, 5000, 17)
    yq, yk = dk.rotary(rope, i32(positions), q, k, q_out=q, k_out=k)
    assert yq.data_ptr() == q.data_ptr() and yk.data_ptr() == k.data_ptr()
    check_turned(rope, q, xq, positions, "f32")
    check_turned(rope, k, xk, positions, "f32")
    dk.rotary(rope, i32(-positions), q, q_out=q)
    # two turns, each off by 16 half-steps of the largest element
    assert np.abs(q.double().cpu().numpy() - xq).max() <= 34 * 2.0 ** -24 * np.abs(xq).max()


def test_rotary_leaves_what_lies_around(dk):
    """A strided output: the elements between its heads stay."""
    rng = np.random.default_rng(4)
    rope = dk.Rotary(32)
    q, x = heads(rng, 6, 2, 64, "bf16", "plain")
    wide = torch.full((6, 5, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    positions = rng.integers(0, 99, 6)
    out, _ = dk.rotary(rope, i32(positions), q, q_out=wide[:, 1:3])
    check_turned(rope, out, x, positions, "bf16")
    assert (wide[:, 0] == 9).all() and (wide[:, 3:] == 9).all()


def test_rotary_of_nothing_and_on_a_stream(dk):
    rope = dk.Rotary(64)
    none = torch.empty((0, 4, 64), dtype=torch.float16, device=DEV)
    assert dk.rotary(rope, i32([]), none)[0].shape == (0, 4, 64)
    no_heads = torch.empty((3, 0, 64), dtype=torch.float16, device=DEV)
    q, x = heads(np.random.default_rng(0), 3, 2, 64, "f16", "plain")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, nothing = dk.rotary(rope, i32([1, 2, 3]), q, no_heads, stream=s)
    s.synchronize()
    assert nothing.shape == (3, 0, 64)
    check_turned(rope, got, x, [1, 2, 3], "f16")


def test_rotary_passes_infinities_and_nan(dk):
    """A bad element reaches its own pair only."""
    rope = dk.Rotary(64)
    q = torch.ones(1, 2, 64, device=DEV)
    q[0, 0, 3], q[0, 1, 40] = float("nan"), float("inf")
    y, _ = dk.rotary(rope, i32([5]), q)
    bad = ~torch.isfinite(y[0])
    want = torch.zeros(2, 64, dtype=torch.bool, device=DEV)
    want[0, [3, 35]], want[1, [8, 40]] = True, True
    assert torch.equal(bad, want)


def test_rotary_refusals(dk):
    rope = dk.Rotary(64)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    at = i32([0, 1, 2])
    bad = [
        lambda: dk.rotary(None, at, q), lambda: dk.rotary(rope, at.long(), q),
        lambda: dk.rotary(rope, at[:2], q), lambda: dk.rotary(rope, at, q[..., :62]),
        lambda: dk.rotary(rope, at, q.double()), lambda: dk.rotary(rope, at, q, q.float()),
        lambda: dk.rotary(rope, at, q, q[:2]), lambda: dk.rotary(rope, at, q.transpose(1, 2)),
        lambda: dk.rotary(rope, at, q, k_out=q), lambda: dk.rotary(rope, at, q, q_out=q[:, :2]),
        lambda: dk.rotary(rope, at, q, q_out=q[:, :1].expand(3, 4, 64)),
        lambda: dk.rotary(rope, at, q, q_out=q.view(4, 3, 64).transpose(0, 1)),
        lambda: dk.rotary(rope, at.cpu(), q), lambda: dk.rotary(rope, at, q.cpu()),
        lambda: dk.rotary(rope, at, torch.zeros(3, 1, 1026, device=DEV)),
    ]
    for call in bad:
        with pytest.raises((TypeError, ValueError, dk.DcpError)):
            call()

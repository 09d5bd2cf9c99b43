"""Attention over whole prompts on the GPU against its definition in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import prompt_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative


@pytest.fixture(scope="module")
def dk():
    import sparse_attention_indexer_stable_gb300 as dk
    return dk


def inputs(seed, rows, heads, group, dim, dtype, layout="fused", size=1.5):
    """q, k, v as a user has them."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        x = torch.randn(*shape, generator=g, device=DEV)
        return x * torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=DEV))

    hq = heads * group
    x = normal(rows, hq + 2 * heads, dim)
    x[:, :hq] *= size
    x = x.to(TYPES[dtype])
    if layout == "odd":  # no 16-byte accesses
        flat = torch.zeros(rows * (hq + 2 * heads) * (dim + 3) + 1, dtype=x.dtype, device=DEV)[1:]
        wide = flat.view(rows, hq + 2 * heads, dim + 3)[..., 1:1 + dim]
        wide.copy_(x)
        x = wide
    parts = [x[:, :hq], x[:, hq:hq + heads], x[:, hq + heads:]]
    if layout == "plain":
        parts = [t.contiguous() for t in parts]
    if layout == "heads first":
        parts = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in parts]
    return parts


def bounds(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int64)


def check(dk, q, k, v, starts, dtype, **kw):
    """One call against the definition, and the rows of no sequence left alone."""
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    got, got_lse = dk.prompt_attention(q, k, v, torch.tensor(starts, device=DEV).int(), out=out,
                                       lse=lse, **kw)
    assert got.data_ptr() == out.data_ptr() and got_lse.data_ptr() == lse.data_ptr()
    want, want_lse, tol, lse_tol = ref.attention(q, k, v, starts, p_step=STEP[dtype], **kw)
    none = torch.isnan(want_lse)
    assert (out[none] == 7).all() and (lse[none] == 7).all()
    ok = ~none
    err = (out[ok].double() - want[ok]).abs()
    assert not torch.isnan(out[ok]).any() and not torch.isnan(lse[ok]).any()
    room = tol[ok] + STEP[dtype] * (1 + 2.0 ** -8) * want[ok].abs() + 2.0 ** -25
    assert (err <= room).all(), float((err - room).max())
    assert ((lse[ok].double() - want_lse[ok]).abs() <= lse_tol[ok]).all()
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,heads,group", [
    ([1], 1, 1), ([2, 1, 3], 2, 4), ([127], 1, 8), ([128], 2, 2), ([129, 0, 64], 1, 7),
    ([257, 31], 1, 3), ([0, 0, 5], 3, 1), ([600], 1, 16), ([33, 500, 1, 260], 2, 8)])
def test_matches_the_definition(dk, dtype, dim, lens, heads, group):
    q, k, v = inputs(sum(lens) + dim, sum(lens), heads, group, dim, dtype)
    check(dk, q, k, v, bounds(lens), dtype)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kw", [
    dict(causal=False), dict(window=1), dict(window=40), dict(window=128), dict(window=333),
    dict(causal=False, window=70), dict(softcap=5.0), dict(softcap=30.0, window=200, scale=0.3),
    dict(scale=-0.07), dict(scale=1e-30), dict(softcap=1e-30), dict(softcap=1e30)])
def test_masks_scales_and_caps(dk, dim, kw):
    lens = [190, 3, 700]
    for dtype in ("bf16", "f16"):
        q, k, v = inputs(7, sum(lens), 2, 4, dim, dtype)
        check(dk, q, k, v, bounds(lens), dtype, **kw)


@pytest.mark.parametrize("layout", ["plain", "odd", "heads first"])
@pytest.mark.parametrize("dim,group", [(64, 5), (128, 1), (128, 12), (256, 6)])
def test_layouts(dk, layout, dim, group):
    lens = [140, 17, 300]
    q, k, v = inputs(3, sum(lens), 2, group, dim, "bf16", layout)
    check(dk, q, k, v, bounds(lens), "bf16")


@pytest.mark.parametrize("group", [17, 24, 64, 96, 128, 130])
def test_many_heads_share_a_key(dk, group):
    q, k, v = inputs(group, 150, 1, group, 64, "bf16")
    check(dk, q, k, v, [0, 70, 150], "bf16")


def test_one_head_and_row_strides_of_no_meaning(dk):
    """Dimensions of one element have any stride."""
    q, k, v = inputs(5, 1, 1, 1, 128, "bf16", "plain")
    strided = [t.as_strided((1, 1, 128), (3, 5, 1)) for t in (q, k, v)]
    check(dk, *strided, [0, 1], "bf16")
    q, k, v = inputs(6, 40, 1, 1, 128, "bf16", "plain")
    check(dk, *[t.as_strided((40, 1, 128), (128, 3, 1)) for t in (q, k, v)], [0, 40], "bf16")


def test_shared_rows(dk):
    """Keys and values broadcast over rows and heads (strides of 0)."""
    q, k, v = inputs(8, 200, 4, 2, 64, "f16", "plain")
    k, v = k[:, :1].expand(200, 4, 64), v[:1].expand(200, 4, 64)
    check(dk, q, k, v, [0, 200], "f16")


def test_rows_of_no_sequence_are_left_and_their_values_do_not_matter(dk):
    """Rows before the first and behind the last sequence: NaN in all inputs."""
    for dim in (64, 128, 256):
        q, k, v = [t.clone() for t in inputs(9, 500, 2, 4, dim, "bf16")]
        for t in (q, k, v):
            t[:37], t[411:] = float("nan"), float("inf")
        check(dk, q, k, v, [37, 150, 150, 411], "bf16")
        check(dk, q, k, v, [37, 150, 411], "bf16", causal=False)


def test_starts_outside_the_rows_are_cut(dk):
    q, k, v = inputs(10, 300, 1, 4, 64, "bf16")
    out, lse = dk.prompt_attention(q, k, v, torch.tensor([-5, 100, 900], device=DEV).int())
    want, want_lse = dk.prompt_attention(q, k, v, torch.tensor([0, 100, 300], device=DEV).int())
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # no order: any result, but nothing is touched outside
    for starts in ([200, 10, 250, -3, 2 ** 31 - 1], [0, 300, 5], [300, 0], [10, 290, 0, 300, 1]):
        for causal in (True, False):
            dk.prompt_attention(q, k, v, torch.tensor(starts, device=DEV).int(), causal=causal)
    torch.cuda.synchronize()
    again, again_lse = dk.prompt_attention(q, k, v, torch.tensor([0, 100, 300], device=DEV).int())
    assert torch.equal(again, want) and torch.equal(again_lse, want_lse)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("where", ["v", "k"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_has_no_influence(dk, dim, where, value):
    """A bad key or value at row 203 of a sequence: earlier rows, and rows whose
    window has passed it, are as without it; the others that see it are not."""
    q, k, v = [t.clone() for t in inputs(12, 420, 2, 4, dim, "bf16")]
    starts = torch.tensor([0, 20, 420], device=DEV).int()
    for kw in (dict(), dict(window=90)):
        plain, plain_lse = dk.prompt_attention(q, k, v, starts, **kw)
        kept = {"k": k, "v": v}[where][223].clone()
        {"k": k, "v": v}[where][223, :, dim // 2] = value
        out, lse = dk.prompt_attention(q, k, v, starts, **kw)
        {"k": k, "v": v}[where][223] = kept
        sees = torch.zeros(420, dtype=torch.bool, device=DEV)
        sees[223:min(420, 223 + kw.get("window", 420))] = True
        # rows that were computed another way than in the call without it
        # differ by both calls' roundings
        _, _, tol, lse_tol = ref.attention(q, k, v, starts.tolist(), **kw)
        room = 2 * tol + 2.0 ** -7 * plain.double().abs()
        near = (out.double() - plain.double()).abs() <= room
        assert near[~sees].all()
        assert ((lse - plain_lse).double().abs() <= 2 * lse_tol)[~sees].all()
        if where == "v":
            assert ((lse - plain_lse).double().abs() <= 2 * lse_tol).all()
            assert near[..., :dim // 2].all() and near[..., dim // 2 + 1:].all()
            seen = out[sees][..., dim // 2].float()
            # a probability of this token that rounds to 0 would give NaN for
            # infinities; scores here are far from that
            assert torch.isnan(seen).all() if math.isnan(value) else (seen == value).all()
        elif math.isnan(value):
            assert torch.isnan(out[sees].float()).all() and torch.isnan(lse[sees]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_light_tokens_beside_a_heavy_one(dk, dtype):
    """One score far above thousands of equal ones: their sum counts."""
    n, gap = 6000, 16.0
    q = torch.zeros(n, 1, 64, device=DEV)
    k = torch.zeros(n, 1, 64, device=DEV)
    v = torch.zeros(n, 1, 64, device=DEV)
    q[:, 0, 0] = 1.0
    k[17, 0, 0] = gap  # weight e^16 of the others'
    v[:, 0, 1], v[17, 0, 1], v[17, 0, 2] = 1.0, 0.0, 1.0
    q, k, v = (t.to(TYPES[dtype]) for t in (q, k, v))
    check(dk, q, k, v, [0, n], dtype, scale=1.0)


def test_a_heavy_token_late(dk):
    """The maximum grows by leaps along the row: every sum so far is shrunk."""
    n = 1500
    for dim in (64, 128, 256):
        q, k, v = [t.clone() for t in inputs(13, n, 1, 2, dim, "f16")]
        q[..., 0] = 1.0
        k[:, 0, 0] = torch.linspace(0, 300, n, device=DEV) * dim ** 0.5 / 8
        check(dk, q, k, v, [0, n], "f16")


def test_huge_scores_stay_finite(dk):
    """Scores far beyond the exponent's range on both sides."""
    for dim in (64, 128, 256):
        q, k, v = inputs(14, 300, 1, 4, dim, "bf16", size=300.0)
        out, lse = dk.prompt_attention(q, k, v, torch.tensor([0, 300], device=DEV).int(),
                                       scale=40.0)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


def test_minus_infinity_as_a_score(dk):
    """Keys at -infinity weigh nothing; a row that sees only such gives zeros."""
    q = torch.ones(130, 1, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(130, 1, 64, dtype=torch.bfloat16, device=DEV)
    v = torch.ones(130, 1, 64, dtype=torch.bfloat16, device=DEV)
    k[:5, 0, 0] = -float("inf")
    out, lse = dk.prompt_attention(q, k, v, torch.tensor([0, 130], device=DEV).int())
    assert (out[:5] == 0).all() and (lse[:5] == -float("inf")).all()
    assert (out[5:] == 1).all()
    want = 8.0 + torch.log(torch.arange(1, 126, device=DEV).double())
    assert ((lse[5:, 0].double() - want).abs() <= 2.0 ** -18).all()


def test_deterministic(dk):
    lens = [1000, 7, 400, 90]
    q, k, v = inputs(15, sum(lens), 2, 8, 128, "bf16")
    starts = torch.tensor(bounds(lens), device=DEV).int()
    first = dk.prompt_attention(q, k, v, starts)
    for _ in range(5):
        again = dk.prompt_attention(q, k, v, starts)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_in_a_graph_with_other_lengths(dk):
    """A captured call is replayed over other sequences of the same batch."""
    q, k, v = inputs(16, 600, 2, 4, 128, "bf16")
    starts = torch.tensor([0, 200, 400, 600], device=DEV).int()
    out, lse = torch.zeros_like(q.contiguous()), torch.zeros(600, 8, device=DEV)
    dk.prompt_attention(q, k, v, starts, out=out, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dk.prompt_attention(q, k, v, starts, out=out, lse=lse)
    for cut in ([0, 600, 600, 600], [0, 1, 2, 599], [5, 130, 400, 555]):
        starts.copy_(torch.tensor(cut))
        out.fill_(7), lse.fill_(7)
        graph.replay()
        want, want_lse = torch.full_like(out, 7), torch.full_like(lse, 7)
        dk.prompt_attention(q, k, v, starts, out=want, lse=want_lse)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_calls_at_once(dk):
    sets = [inputs(20 + i, 900, 2, 8, d, "bf16") for i, d in enumerate((128, 64))]
    starts = torch.tensor([0, 333, 900], device=DEV).int()
    want = [dk.prompt_attention(*s, starts) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(dk.prompt_attention(*sets[i], starts, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_many_short_sequences(dk):
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 12, 3000)
    q, k, v = inputs(17, int(lens.sum()), 1, 4, 64, "bf16")
    starts = bounds(lens)
    out, lse = dk.prompt_attention(q, k, v, torch.tensor(starts, device=DEV).int())
    # a sample of them by the definition
    for b in rng.integers(0, 3000, 40):
        a, e = int(starts[b]), int(starts[b + 1])
        if a == e:
            continue
        want, want_lse, tol, lse_tol = ref.attention(q[a:e], k[a:e], v[a:e], [0, e - a])
        assert ((out[a:e].double() - want).abs() <= tol + 2.0 ** -7 * want.abs()).all()
        assert ((lse[a:e].double() - want_lse).abs() <= lse_tol).all()
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dim,heads,group", [(64, 8, 1), (128, 8, 8), (256, 4, 2)])
def test_more_work_than_the_gpu_holds(dk, dim, heads, group):
    """Every CTA takes several units, of all lengths."""
    lens = [1100, 3, 260, 700, 0, 41, 900, 129, 513]
    q, k, v = inputs(21, sum(lens), heads, group, dim, "bf16")
    check(dk, q, k, v, bounds(lens), "bf16")
    check(dk, q, k, v, bounds(lens), "bf16", window=200)


def test_nothing_to_do(dk):
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = dk.prompt_attention(q, k, k, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    q, k, v = inputs(18, 30, 1, 2, 64, "bf16")
    out = torch.full((30, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    for starts in ([3], [0, 0, 0], [30, 30]):
        dk.prompt_attention(q, k, v, torch.tensor(starts, device=DEV).int(), out=out)
    assert (out == 7).all()


def test_refusals(dk):
    q, k, v = inputs(19, 30, 2, 3, 64, "bf16", "plain")
    starts = torch.tensor([0, 30], device=DEV).int()
    bad = [
        (q.float(), k, v, starts, {}), (q, k.half(), v, starts, {}), (q, k, v.cpu(), starts, {}),
        (q[..., :32], k[..., :32], v[..., :32], starts, {}), (q, k[:20], v[:20], starts, {}),
        (q, k, v[:, :1], starts, {}), (q[:, :5], k, v, starts, {}), (q, k, v, starts.long(), {}),
        (q, k, v, starts[:0], {}), (q, k, v, starts.cpu(), {}), (q, k, v, starts, {"window": -1}),
        (q, k, v, starts, {"scale": float("nan")}), (q, k, v, starts, {"softcap": -2.0}),
        (q, k, v, starts, {"softcap": float("inf")}),
        (q.transpose(1, 2), k, v, starts, {}), (q, k, v, starts, {"out": q[:20]}),
        (q, k, v, starts, {"out": torch.empty(30, 6, 64, device=DEV)}),
        (q, k, v, starts, {"lse": torch.empty(30, 6, dtype=torch.float64, device=DEV)}),
        (q, k, v, starts, {"window": 2 ** 40}), (q[0], k, v, starts, {}),
    ]
    for *args, kw in bad:
        with pytest.raises((TypeError, ValueError, dk.DcpError)):
            dk.prompt_attention(*args, **kw)

"""Attention over prompts at the ends of its inputs' range."""
import pytest

torch = pytest.importorskip("torch")

from . import prompt_reference as ref  # noqa: E402
from .test_gpu_prompt import DEV, STEP, dk, inputs  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# an element of q and of k: their product is the score, up to scale
HUGE = [("f16", e) for e in (2.0 ** 10, 2.0 ** 13, 20000.0, 55072.0, 65504.0)] + [
    ("bf16", e) for e in (2.0 ** 10, 2.0 ** 14, 184320.0, 2.0 ** 23, 2.0 ** 40, 2.0 ** 63)]


def starts_of(*rows):
    return torch.tensor(rows, device=DEV).int()


def near_value(out, v, dtype):
    """Whether out is v where one key has all of the weight: a probability's
    rounding (half a step), the output's, and five of fp32."""
    room = 2.0 * STEP[dtype] * (1 + STEP[dtype]) + 5 * 2.0 ** -24
    return ((out.double() - v.double()).abs() <= room * v.double().abs() + 2.0 ** -25).all()


def near_score(lse, score):
    """The scale, log2 e, their product, the score's, the reference, its sum with
    log2 l, and ln 2 and its product: eight roundings of fp32; log2 l itself."""
    return ((lse.double() - score).abs() <= 2.0 ** -21 * abs(score) + 2.0 ** -19).all()


@pytest.mark.parametrize("dtype,e", HUGE)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_one_key_at_a_huge_score(dk, dtype, e, dim, sign):  # noqa: F811
    for scale in (None, 0.04, -0.05):
        q, k, v = [t.clone() for t in inputs(1, 1, 2, 4, dim, dtype)]
        q.zero_(), k.zero_()
        q[..., 3], k[..., 3] = e, sign * e
        out, lse = dk.prompt_attention(q, k, v, starts_of(0, 1), scale=scale)
        assert near_value(out, v.repeat_interleave(4, 1), dtype)
        e_in = float(q[0, 0, 3])
        assert near_score(lse, sign * e_in * e_in * (dim ** -0.5 if scale is None else scale))


@pytest.mark.parametrize("dtype,e", HUGE)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_key_far_above_the_others(dk, dtype, e, dim):  # noqa: F811
    """Rows behind it give its value; those before it do not notice."""
    n, heavy = 300, 150
    q, k, v = [t.clone() for t in inputs(2, n, 2, 4, dim, dtype, size=0.5)]
    q[..., 0], k[..., 0] = e, 0.0
    k[heavy, :, 0] = e
    out, lse = dk.prompt_attention(q, k, v, starts_of(0, n))
    assert near_value(out[heavy:], v[heavy].repeat_interleave(4, 0), dtype)
    score = float(q[0, 0, 0]) ** 2 * dim ** -0.5
    # the other elements' products: far below a step of the score, or a few units
    assert ((lse[heavy:].double() - score).abs() <= 2.0 ** -20 * score + 64.0).all()
    before, before_lse = dk.prompt_attention(q[:heavy], k[:heavy], v[:heavy], starts_of(0, heavy))
    assert torch.equal(out[:heavy], before) and torch.equal(lse[:heavy], before_lse)


@pytest.mark.parametrize("dtype,e", HUGE)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_huge_scores(dk, dtype, e, dim, sign):  # noqa: F811
    """All keys weigh the same: row i gives the mean of its values."""
    n = 400
    q, k, v = [t.clone() for t in inputs(3, n, 1, 2, dim, dtype)]
    q.zero_(), k.zero_()
    q[..., 1], k[..., 1] = e, sign * e
    out, lse = dk.prompt_attention(q, k, v, starts_of(0, n))
    count = torch.arange(1, n + 1, device=DEV).double()
    mean = (torch.cumsum(v.double(), 0) / count[:, None, None]).repeat_interleave(2, 1)
    size = (torch.cumsum(v.double().abs(), 0) / count[:, None, None]).repeat_interleave(2, 1)
    # all probabilities are rounded alike, half a step; accumulations cut off a
    # bit; the output's rounding
    room = size * (STEP[dtype] * (1 + 2.0 ** -6) + (n / 16 + 32) * 2.0 ** -23)
    room += STEP[dtype] * (1 + 2.0 ** -6) * mean.abs() + 2.0 ** -25
    assert ((out.double() - mean).abs() <= room).all()
    e_in = float(q[0, 0, 1])
    score = sign * e_in * e_in * dim ** -0.5
    want = score + torch.log(count)[:, None]
    assert ((lse.double() - want).abs() <= 2.0 ** -21 * abs(score) + 2.0 ** -18).all()


@pytest.mark.parametrize("dtype,e", [("f16", 40000.0), ("bf16", 2.0 ** 20), ("bf16", 2.0 ** 60)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("order", ["up", "any"])
def test_a_maximum_that_travels(dk, dtype, e, dim, order):  # noqa: F811
    """Keys far apart from each other, from far below 0 to far above: a row gives
    the value of the largest that it sees."""
    n, group = 900, 4
    g = torch.Generator(device=DEV).manual_seed(dim)
    q, k, v = [t.clone() for t in inputs(7, n, 1, group, dim, dtype)]
    q.zero_(), k.zero_()
    place = torch.arange(n, device=DEV)
    if order == "any":
        place = torch.randperm(n, generator=g, device=DEV)
    # two elements, so that each key has a score of its own
    q[..., 0], q[..., 1] = e, e / 256
    k[..., 0] = (e * ((place // 30) / 15.0 - 1.0))[:, None].to(k.dtype)
    k[..., 1] = (e * (place % 30) / 4.0 / 15.0)[:, None].to(k.dtype)
    scores = (q[0, 0].double() * k[:, 0].double()).sum(-1)
    i = torch.arange(n, device=DEV)
    for window in (0, 77):
        sees = i <= i[:, None]
        if window:
            sees &= i > i[:, None] - window
        top = torch.where(sees, scores, -float("inf"))
        best = top.argmax(-1)
        second = top.scatter(-1, best[:, None], -float("inf")).amax(-1)
        alone = (top.amax(-1) - second) * dim ** -0.5 > 1e3  # no other key has any weight
        assert alone.float().mean() > 0.8
        out, lse = dk.prompt_attention(q, k, v, starts_of(0, n), window=window)
        assert near_value(out[alone], v[best][alone].repeat_interleave(group, 1), dtype)
        want = (scores[best] * dim ** -0.5)[alone, None]
        # the sum of two products, and what near_score counts
        size = ((q[0, 0].double() * k[best, 0].double()).abs().sum(-1) * dim ** -0.5)[alone, None]
        assert ((lse[alone].double() - want).abs() <= 2.0 ** -20 * size + 2.0 ** -19).all()


# -------------------------------------------------------------------- caps
def fill_shared_memory(dk, dim, value):  # noqa: F811
    """Leaves `value` as queries in every SM's shared memory."""
    q = torch.full((256 * 64, 8, dim), value, dtype=torch.bfloat16, device=DEV)
    dk.prompt_attention(q, q[:, :1], q[:, :1], starts_of(*range(0, 256 * 64 + 1, 256)))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [3, 7, 1])
@pytest.mark.parametrize("softcap", [0.0, 3.0])
def test_what_shared_memory_held_does_not_matter(dk, dim, group, softcap):  # noqa: F811
    """Groups that leave a tile's last rows empty, with scores on both sides of
    the cap: the same bits each time."""
    q, k, v = inputs(4, 1000, 2, group, dim, "bf16", size=0.1)
    first = None
    for value in (0.0, 300.0, float("nan"), 0.0, 1.0):
        fill_shared_memory(dk, dim, value)
        got = dk.prompt_attention(q, k, v, starts_of(0, 700, 1000), softcap=softcap)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=3.0), dict(softcap=3.0, window=70)])
def test_a_row_does_not_depend_on_others(dk, dim, group, kw):  # noqa: F811
    """The same bits whatever other heads, later tokens and other sequences hold,
    on either side of the cap."""
    n, cut = 500, 333
    q, k, v = [t.clone() for t in inputs(5, n, 2, group, dim, "bf16", size=0.6)]
    want = dk.prompt_attention(q, k, v, starts_of(0, cut, n), **kw)
    # a prompt and its prefix
    part = dk.prompt_attention(q[:cut - 50], k[:cut - 50], v[:cut - 50], starts_of(0, cut - 50),
                               **kw)
    assert all(torch.equal(a[:cut - 50], b) for a, b in zip(want, part))
    # other queries in later rows and behind the sequence
    loud = q.clone()
    loud[200:] *= 50.0
    got = dk.prompt_attention(loud, k, v, starts_of(0, cut, n), **kw)
    assert all(torch.equal(a[:200], b[:200]) for a, b in zip(want, got))
    # other heads
    if group > 1:
        loud = q.clone()
        loud[:, 1::group] *= 50.0
        got = dk.prompt_attention(loud, k, v, starts_of(0, cut, n), **kw)
        assert all(torch.equal(a[:, ::group], b[:, ::group]) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kw", [
    dict(softcap=1e36), dict(softcap=1e37), dict(softcap=1e38), dict(softcap=3e38),
    dict(softcap=1e10, scale=1e-30), dict(softcap=3e38, scale=-0.3), dict(softcap=1.0, scale=2e-38)])
def test_caps_that_are_far_away(dk, dtype, kw):  # noqa: F811
    """As without one."""
    for dim in (64, 128):
        q, k, v = inputs(6, 300, 2, 3, dim, dtype)
        out, lse = dk.prompt_attention(q, k, v, starts_of(0, 300), **kw)
        want, want_lse, tol, lse_tol = ref.attention(q, k, v, [0, 300], p_step=STEP[dtype], **kw)
        assert ((out.double() - want).abs() <= tol + STEP[dtype] * (1 + 2.0 ** -8) * want.abs()
                + 2.0 ** -25).all()
        assert ((lse.double() - want_lse).abs() <= lse_tol).all()

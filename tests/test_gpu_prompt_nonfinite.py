"""Attention over prompts with infinities and NaN among the values: what rows that
see them get, and what they and their neighbours cost."""
import pytest

torch = pytest.importorskip("torch")

from . import prompt_reference as ref  # noqa: E402
from .test_gpu_prompt import DEV, STEP, dk, inputs  # noqa: E402,F401
from .test_gpu_prompt_give_up import attend, lib  # noqa: E402,F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def starts_of(*rows):
    return torch.tensor(rows, device=DEV).int()


def expected(q, k, v, starts, **kw):
    """The definition: finite columns in 64 bits, the others by what the row sees in
    them: NaN with a NaN or both infinities, else the infinity."""
    def part(x):
        return ref.attention(q, k, x, starts, **kw)

    _, lse, _, lse_tol = part(v)
    out, _, tol, _ = part(torch.where(torch.isfinite(v), v, 0))
    sees = [part(x.to(v.dtype))[0] > 0 for x in (torch.isnan(v), v == INF, v == -INF)]
    out = torch.where(sees[1], INF, out)
    out = torch.where(sees[2], -INF, out)
    return torch.where(sees[0] | (sees[1] & sees[2]), NAN, out), lse, tol, lse_tol


def check(dk, q, k, v, starts, dtype, **kw):  # noqa: F811
    out, lse = dk.prompt_attention(q, k, v, starts_of(*starts), **kw)
    want, want_lse, tol, lse_tol = expected(q, k, v, starts, **kw)
    nan, inf = torch.isnan(want), torch.isinf(want)
    assert torch.equal(torch.isnan(out), nan)
    assert (out.double() == want)[inf].all()
    ok = ~nan & ~inf
    room = tol + STEP[dtype] * (1 + 2.0 ** -8) * want.abs() + 2.0 ** -25
    assert ((out.double() - want).abs() <= room)[ok].all()
    assert ((lse.double() - want_lse).abs() <= lse_tol).all()


# (row, column, value) of what is not finite
PLACES = {
    "first": [(0, 0, INF)],
    "nan first": [(0, 5, NAN)],
    "both signs": [(3, 9, INF), (170, 9, -INF), (400, 9, INF), (2, 1, -INF)],
    "infinity, then nan": [(130, 7, INF), (420, 7, NAN), (421, 8, NAN)],
    "late": [(590, 0, INF), (599, 1, NAN)],
    "everywhere": [(r, r % 64, INF) for r in range(0, 600, 37)],
    "whole row": [(260, c, NAN) for c in range(64)],
}


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("place", sorted(PLACES))
@pytest.mark.parametrize("kw", [dict(), dict(window=150), dict(causal=False), dict(softcap=4.0)])
def test_rows_get_what_they_see(dk, dim, place, kw):  # noqa: F811
    for dtype, group in (("bf16", 4), ("f16", 3)):
        # scores close together: no probability rounds to 0
        q, k, v = [t.clone() for t in inputs(1, 640, 2, group, dim, dtype, size=0.02)]
        for r, c, x in PLACES[place]:
            v[20 + r, :, c + dim - 64] = x
        v[:20], v[620:] = NAN, INF
        check(dk, q[20:620], k[20:620], v[20:620], [0, 350, 600], dtype, **kw)
        if not kw:
            out, _ = dk.prompt_attention(q, k, v, starts_of(20, 370, 620))
            alone, _ = dk.prompt_attention(q[20:620], k[20:620], v[20:620], starts_of(0, 350, 600))
            assert torch.equal(out[20:620].nan_to_num(7.0), alone.nan_to_num(7.0))


def test_large_values_beside_infinite_ones(dk):  # noqa: F811
    """Values that the running sum overflows with, in rows that see an infinity in
    another column."""
    n = 700
    q, k, v = [t.clone() for t in inputs(2, n, 1, 4, 128, "bf16", size=0.02)]
    q[..., 0] = 8.0
    k[..., 0] = torch.linspace(0, 50, n, device=DEV)[:, None]  # scores to 35, references behind
    v[..., 70:] = 1e30
    v[5, :, 3], v[300, :, 4] = INF, NAN
    check(dk, q, k, v, [0, n], "bf16")


@pytest.mark.parametrize("dim,heads,group", [(64, 8, 4), (128, 8, 8), (256, 2, 4)])
@pytest.mark.parametrize("row,value", [(0, INF), (0, NAN), (1500, NAN)])
def test_a_value_that_rows_see_costs_little(dk, dim, heads, group, row, value):  # noqa: F811
    """Rows that see a value have it from the tensor cores.  Up to 128 tokens before
    it share a step with it and are computed again: 32 rows of a warp in turn, 47
    blocks of 32 keys each, at 5 us a block 7.5 ms beside 0.044."""
    q, k, v = [t.clone() for t in inputs(3, 2048, heads, group, dim, "bf16", size=0.02)]
    starts = starts_of(0, 2048)
    plain = time_of(lambda: dk.prompt_attention(q, k, v, starts))
    v[row, :, 0] = value
    bad = time_of(lambda: dk.prompt_attention(q, k, v, starts))
    assert bad <= (10 if row == 0 else 400) * plain


def time_of(f):
    f()
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[2]


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_behind_the_last_sequence_cost_nothing(dk, dim):  # noqa: F811
    """A padded batch whose padding is NaN takes as long as one of zeros."""
    lens = [257 + 17 * i for i in range(64)]
    starts = starts_of(0, *torch.cumsum(torch.tensor(lens), 0).tolist())
    q, k, v = [t.clone() for t in inputs(4, sum(lens) + 200, 2, 7, dim, "bf16")]
    times = []
    for value in (0.0, NAN, 0.0, NAN):
        for t in (q, k, v):
            t[sum(lens):] = value
        # and queries of it in shared memory, in the rows that 7 heads leave empty
        x = torch.full((16384, 8, dim), value, dtype=torch.bfloat16, device=DEV)
        cut = starts_of(*range(0, 16385, 256))
        one = []
        for _ in range(7):
            dk.prompt_attention(x, x[:, :1], x[:, :1], cut)
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            dk.prompt_attention(q, k, v, starts)
            b.record()
            torch.cuda.synchronize()
            one.append(a.elapsed_time(b))
        times.append(min(one))
    assert times[1] + times[3] <= 1.1 * (times[0] + times[2])


def test_long_rows_that_are_computed_again(lib, dk):  # noqa: F811
    """An infinity in the last value of a long prompt: the rows of its tile do not
    see it and are computed again, for longer than the patience of the waits for
    them (2 ms in the race-check build)."""
    n = 256 * 120 + 3
    q, k, v = [t.clone() for t in inputs(5, n, 4, 1, 128, "bf16")]
    plain, plain_lse = dk.prompt_attention(q, k, v, starts_of(0, n))
    v[n - 1, :, 3] = INF
    lib.dcp_prompt_selftest_withhold(-1, -1, -1)
    out, lse, status = attend(lib, q, k, v, starts_of(0, n))
    assert status == 0
    assert torch.isfinite(lse).all() and torch.isfinite(out[:-1]).all()
    assert (out[-1, :, 3] == INF).all() and torch.isfinite(out[-1, :, 4:]).all()
    assert torch.equal(out[:256 * 120], plain[:256 * 120])
    got, got_lse = dk.prompt_attention(q, k, v, starts_of(0, n))
    assert torch.equal(out, got) and torch.equal(lse, got_lse)
    # the same row both ways: half a step of the output's and of the probabilities'
    # rounding, of values up to 8
    assert (out[-3:-1] - plain[-3:-1]).abs().max() <= 2.0 ** -4

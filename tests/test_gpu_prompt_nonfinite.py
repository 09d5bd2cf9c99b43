"""Attention over prompts with infinities and NaN among the inputs: what they cost
the rows that do not see them."""
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_prompt import DEV, dk, inputs  # noqa: E402,F401
from .test_gpu_prompt_give_up import attend, lib  # noqa: E402,F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def starts_of(*rows):
    return torch.tensor(rows, device=DEV).int()


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
        times.append(sorted(one)[3])
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

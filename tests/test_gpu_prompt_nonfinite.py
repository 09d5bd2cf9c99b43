"""Attention over prompts with infinities and NaN among the inputs: what they cost
the rows that do not see them."""
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_prompt import DEV, dk, inputs  # noqa: E402,F401

pytestmark = pytest.mark.gpu

NAN = float("nan")


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

"""kv4_extend with as many sequences as it takes, lengths and the list's count in
place: the CTAs of a cluster, each with all of the shared memory that it may have."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import prompt_reference as ref  # noqa: E402
from .test_gpu_batch import DEV, batch, dk, i32  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,extra", [(1, 0), (9, 5)])
def test_extend_in_place_with_the_most_sequences(dk, most, extra):  # noqa: F811
    B = 16384
    rng = np.random.default_rng(most)
    table, lens, counts, free, pages = batch(rng, B, 16, 100, most)
    places = int(counts.sum()) + extra
    t, n, u = i32(table), i32(lens), i32([0])
    step = dk.Kv4Step(torch.empty(places, dtype=torch.int64, device=DEV), *[
        torch.empty(places, dtype=torch.int32, device=DEV) for _ in range(3)],
        torch.empty(B + 1, dtype=torch.int32, device=DEV), n, u)
    dk.kv4_extend(t, n, i32(counts), i32(free), u, places, 16, pages, out=step)
    want = ref.extend(table, lens, counts, free, 0, places, 16, pages)
    assert [x.tolist() for x in step] == list(want[:7]) and t.tolist() == want[7]

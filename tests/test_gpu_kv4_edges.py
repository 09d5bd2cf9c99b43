"""Edges of the 4-bit cache's operators on the GPU."""
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

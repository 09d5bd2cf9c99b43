"""Prompts and rotary positions in tensors whose elements lie beyond 32 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import prompt_reference as ref  # noqa: E402
from .test_gpu_batch import check_turned, i32  # noqa: E402
from .test_gpu_prompt import DEV, STEP, dk, inputs  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,heads,group", [(128, 8, 8), (64, 16, 8)])
def test_the_far_end_of_a_large_batch(dk, dim, heads, group):  # noqa: F811
    width = (heads * group + 2 * heads) * dim
    rows = 2 ** 32 // width + 3000
    last = 700
    fused = torch.empty(rows, heads * group + 2 * heads, dim, dtype=torch.bfloat16, device=DEV)
    assert (rows - last) * heads * group * dim >= 2 ** 31
    fused[-last:] = torch.cat(inputs(3, last, heads, group, dim, "bf16"), 1)
    q, k, v = fused.split([heads * group, heads, heads], 1)
    out = torch.empty(rows, heads * group, dim, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(rows, heads * group, device=DEV)
    out[-last - 5:], lse[-last - 5:] = 7.0, 7.0
    cut = [rows - last, rows - 450, rows - 450, rows]
    dk.prompt_attention(q, k, v, i32(cut), out=out, lse=lse)
    assert (out[-last - 5:-last] == 7).all()
    far = [t[-last:] for t in (q, k, v)]
    want, want_lse, tol, lse_tol = ref.attention(*far, [0, last - 450, last - 450, last])
    err = (out[-last:].double() - want).abs()
    assert (err <= tol + STEP["bf16"] * (1 + 2.0 ** -8) * want.abs()).all()
    assert ((lse[-last:].double() - want_lse).abs() <= lse_tol).all()

    # rotary positions, in place; the rows before stay
    positions = torch.zeros(rows, dtype=torch.int32, device=DEV)
    at = np.random.default_rng(0).integers(0, 100000, 40)
    positions[-40:] = i32(at)
    near = fused[rows // 2].clone()
    x = far[0][-40:].double().cpu().numpy()
    rope = dk.Rotary(dim)
    dk.rotary(rope, positions, q, k, q_out=q, k_out=k)
    assert torch.equal(fused[rows // 2].nan_to_num(), near.nan_to_num())
    check_turned(rope, q[-40:], x, at, "bf16")

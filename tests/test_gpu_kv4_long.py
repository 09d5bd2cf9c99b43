"""Attention over long rows whose probabilities differ widely, against closed
forms in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from .test_gpu_kv4 import DEV, dk, i32  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_ids", [False, True])
def test_one_heavy_token_among_many_light_ones(dk, with_ids):  # noqa: F811
    """Light tokens of 2^-25 of the heavy one's probability each, 2^17 of them,
    in rows that one warp walks from end to end: a third of a percent together,
    and all their values on one side."""
    n, page, heads, dim, rows = 131072, 64, 8, 64, 304
    cache = dk.Kv4Cache.allocate(n // page, page, heads, dim, DEV)
    cache.k_scales.fill_(0x38)  # 1
    cache.v_scales.fill_(0x38)
    cache.v_codes.fill_(0x55)   # 3 everywhere
    heavy = (77777 // page, 77777 % page)
    cache.k_codes[heavy][:, 0] = 7  # 6 in the first element, the others' keys are 0
    cache.v_codes[heavy] = 0xDD     # -3
    gen = torch.Generator(device=DEV).manual_seed(1)
    order = torch.randperm(n, generator=gen, device=DEV, dtype=torch.int32)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)
    first = 23.296875
    q = torch.randn(rows, heads, dim, generator=gen, device=DEV).half()
    q[:, :, 0] = first
    out, lse = dk.kv4_attention(cache, q, table.expand(rows, -1), i32([n] * rows),
                                ids=order.expand(rows, -1) if with_ids else None)
    score = 6 * first * dim ** -0.5
    want_lse = score + math.log1p((n - 1) * math.exp(-score))
    light = (n - 1) * math.exp(-want_lse)
    want = 3 * light - 3 * (1 - light)
    assert 0.003 < light < 0.004
    # fp16's rounding of the heavy probability and of the output, the light
    # ones' to fp16's smallest step below a reference of 2^7, and fp32's
    tol = 3 * (2.0 ** -11 + n * 2.0 ** -32 + 2.0 ** -18) + 2.0 ** -11 * abs(want)
    assert np.abs(out.double().cpu().numpy() - want).max() <= tol
    # light tokens beside a heavy one in a lane's running sum count, too
    assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 2.0 ** -18

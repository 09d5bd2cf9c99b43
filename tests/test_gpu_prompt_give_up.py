"""A copy that never lands, in attention over prompts: the CTA that waits for it
gives up, reports it, and leaves NaN for the units that it had not finished; the
rest is right, and so is the next call.

The race-check build of the library leaves a copy out when it is told to: its
barrier is armed and nothing comes, so the waits run out (after about 2 ms there),
and nothing faults.
"""
import ctypes
import time

import pytest

torch = pytest.importorskip("torch")

from sparse_attention_indexer_stable_gb300 import _build  # noqa: E402

from .test_gpu_prompt import dk, inputs  # noqa: E402,F401
from .test_prompt_capi import PROMPT  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(_build.build_race_check())
    P = ctypes.c_void_p
    lib.dcp_prompt_attention.argtypes = [P, P]
    lib.dcp_topk_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.dcp_prompt_selftest_withhold.argtypes = [ctypes.c_int] * 3
    lib.dcp_prompt_selftest_withhold.restype = None
    yield lib
    lib.dcp_prompt_selftest_withhold(-1, -1, -1)


def attend(lib, q, k, v, starts):
    """One call through the C ABI; (out, lse, the device's status)."""
    rows, heads, dim = q.shape
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=q.device)
    lse = torch.full((rows, heads), 7.0, device=q.device)
    args = PROMPT.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), q.stride(1),
                       k.stride(0), k.stride(1), v.stride(0), v.stride(1), starts.data_ptr(),
                       out.data_ptr(), lse.data_ptr(), rows, 1, heads, k.shape[1], dim,
                       len(starts) - 1, 1, 0, 0.0, 0.0)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.dcp_prompt_attention(args, stream) == 0
    status = ctypes.c_uint(0)
    assert lib.dcp_topk_device_status(ctypes.byref(status)) == 0  # waits for the device
    return out, lse, status.value


@pytest.mark.parametrize("dim,group,copy", [
    (64, 4, 0), (64, 4, 3), (128, 4, 0), (128, 4, 1), (128, 4, 4), (256, 2, 0), (256, 2, 2),
    (256, 2, 5)])
@pytest.mark.parametrize("unit", [0, 1])
def test_a_copy_that_never_lands(lib, dk, dim, group, copy, unit):  # noqa: F811
    n = 2600  # with 16 heads several units for every CTA
    q, k, v = inputs(dim, n, 16, group, dim, "bf16")
    starts = torch.tensor([0, n], device="cuda").int()
    want, want_lse = dk.prompt_attention(q, k, v, starts)
    lib.dcp_prompt_selftest_withhold(-1, -1, -1)
    out, lse, status = attend(lib, q, k, v, starts)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)

    lib.dcp_prompt_selftest_withhold(0, unit, copy)
    torch.cuda.synchronize()
    start = time.perf_counter()
    out, lse, status = attend(lib, q, k, v, starts)
    took = time.perf_counter() - start
    # the wait that runs out and those for what is in flight: some of 2 and 4 ms
    assert status == dk.DCP_DEVICE_COPY_TIMEOUT and took < 0.2
    lost = torch.isnan(lse)
    # a unit of each tile's rows, or with it the one that was on its way
    rows = (2 if dim < 256 else 1) * 128
    assert rows // 2 <= int(lost.sum()) <= 3 * rows
    assert torch.isnan(out[lost]).all()
    assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])

    lib.dcp_prompt_selftest_withhold(-1, -1, -1)
    out, lse, status = attend(lib, q, k, v, starts)
    assert status == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)

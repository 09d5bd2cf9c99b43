"""Outputs of attention over prompts that share memory with its inputs are refused."""
import pytest

import sparse_attention_indexer_stable_gb300 as dk

from .test_prompt_capi import prompt

# addresses that are never read: every call is refused.  3 rows of 4 query heads
# and one key/value head of 128, 2 bytes each
Q, KV, LSE = 3 * 4 * 256, 3 * 256, 3 * 4 * 4
APART = dict(q=0x10000, k=0x20000, v=0x30000, starts=0x40000, out=0x50000, lse=0x60000)


@pytest.mark.parametrize("change", [
    dict(out=0x10000), dict(out=0x10000 + Q - 16), dict(out=0x10000 - Q + 16),
    dict(out=0x20000), dict(out=0x20000 + KV - 16), dict(out=0x30000 - Q + 16),
    dict(lse=0x10000 + 512), dict(lse=0x20000 - 4), dict(lse=0x30000 + KV - 4),
    dict(out=0x40000), dict(lse=0x40004), dict(lse=0x50000 + Q - 4), dict(lse=0x50000 - LSE + 4),
    # between the rows of a wider buffer, which it reaches at its end or its beginning
    dict(q_row=4096, out=0x10000 + 8192 - Q + 16), dict(q_row=4096, lse=0x10000 + 8192 - 4),
    # head after head: 3 rows of head 2
    dict(q_row=128, q_head=1024, lse=0x10000 + 2 * 2048 + 512 - 4),
])
def test_outputs_over_inputs(change):
    a = dict(APART)
    a.update(change)
    assert dk.library().dcp_prompt_attention(prompt(**a), None) == dk.DCP_ERR_INVALID


@pytest.mark.gpu
def test_outputs_beside_inputs():
    """The same buffer, with no element in common."""
    torch = pytest.importorskip("torch")
    g = torch.Generator(device="cuda").manual_seed(0)
    starts = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    whole = torch.randn(2, 40, 64, generator=g, device="cuda").bfloat16()
    q, k, v = whole[:, :4], whole[:, 4:6], whole[:, 6:8]
    want, want_lse = dk.prompt_attention(q, k, v, starts)
    out = whole[0, 10:18].view(2, 4, 64)
    lse = whole[0, 20].view(torch.float32)[:8].view(2, 4)
    got, got_lse = dk.prompt_attention(q, k, v, starts, out=out, lse=lse)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    for bad in (whole[0, :8], whole.flatten(0, 1)[34:42]):
        with pytest.raises(dk.DcpError):
            dk.prompt_attention(q, k, v, starts, out=bad.view(2, 4, 64))
    with pytest.raises(dk.DcpError):
        dk.prompt_attention(q, k, v, starts, lse=whole[1, 3].view(torch.float32)[24:].view(2, 4))

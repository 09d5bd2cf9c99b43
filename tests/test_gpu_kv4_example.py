"""The example's decode loop: top-K ids, cache, attention, eviction together."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import kv4_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import sparse_decode
    finally:
        sys.path.pop(0)
    return sparse_decode


def test_decode_loop_against_the_definition(example):
    """Steps across two evictions; every step's attention against 64 bits, over
    a model of the sequences kept on the host."""
    rows, heads, group, dim, limit = 3, 2, 4, 64, 64
    s = example.Sequences(rows, limit, page_size=8, heads=heads, group=group, dim=dim, dcp=2,
                          top_k=24, budget=40, sinks=2, recent=8, seed=5)
    kv = [[] for _ in range(rows)]       # the tokens that each sequence holds
    weights = np.zeros((rows, limit))
    tol = np.zeros((rows, limit))
    evictions = 0
    for step in range(100):
        if s.longest == limit:
            before = s.weights.cpu().numpy()
            assert np.all(np.abs(before - weights) <= tol + 1e-6 * weights)
            kept = s.evict().cpu().numpy()
            evictions += 1
            weights = np.zeros((rows, limit))
            for b in range(rows):
                want = ref.evict(limit, before[b], 40, 2, 8)
                assert np.array_equal(kept[b], want)
                kv[b] = [kv[b][i] for i in want]
                weights[b, :40] = before[b, want]
            tol = np.zeros((rows, limit))
        k, v = (s.normal(rows, heads, dim).bfloat16() for _ in range(2))
        q = (2 * s.normal(rows, heads * group, dim)).bfloat16()
        out, lse, ids = s.step(k, v, q)
        for b in range(rows):
            kv[b].append((k[b].double().cpu().numpy(), v[b].double().cpu().numpy()))
        planes = []
        for i in range(2):
            codes, scales = ref.encode(np.stack([np.stack([t[i] for t in kv[b]])
                                                 for b in range(rows)]))
            planes.append((ref.pack(codes), scales))
        n = s.longest
        # one page per sequence, as long as the sequences are
        host = (planes[0][0], planes[1][0], planes[0][1], planes[1][1])
        want, want_lse, w, out_tol, lse_tol, w_tol = ref.attention(
            host, q.double().cpu().numpy(), np.arange(rows)[:, None], np.full(rows, n),
            ids=ids.cpu().numpy(), positions=limit)
        weights += w
        tol += w_tol + 2.0 ** -22 * (weights + w)
        err = np.abs(out.double().cpu().numpy() - want)
        assert np.all(err <= out_tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -25)
        assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= lse_tol)
    assert evictions == 2


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["sparse_decode.py", "--rows", "2", "--limit", "1280",
                                      "--steps", "3"])
    example.main()
    assert "2 sequences, 4 tokens" in capsys.readouterr().out

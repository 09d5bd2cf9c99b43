"""The example's batches: bookkeeping, rotary positions, cache, attention of
prompts and of the decode steps after them, together."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from . import kv4_reference, prompt_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import prompt_batch
    finally:
        sys.path.pop(0)
    return prompt_batch


class Model:
    """The same engine on the host, by the definitions."""

    def __init__(self, engine, pages, page):
        self.e, self.pages, self.page = engine, pages, page
        self.table, self.lens, self.used = engine.table.tolist(), engine.lens.tolist(), 0
        heads, dim = engine.heads, engine.cache.dim
        # an element may still round to the bf16 next to it, and a code with it:
        # the planes are read from the device, the slots are checked
        self.shape = (pages, page, heads, dim)

    def place(self, counts, places):
        r = ref.extend(self.table, self.lens, counts, list(range(self.pages)), self.used, places,
                       self.page, self.pages)
        self.lens, self.used, self.table = r[5], r[6][0], r[7]
        return r

    def planes(self):
        c = self.e.cache
        return tuple(p.cpu().numpy() for p in (c.k_codes, c.v_codes, c.k_scales, c.v_scales))


def check_turned(e, before, after, positions):
    """q and k of `after` are those of `before`, turned and rounded to bf16."""
    x = before.double().cpu().numpy()
    want = ref.turned(x, positions, e.rope.frequencies)
    size = np.abs(x).max(-1, keepdims=True)
    err = np.abs(after.double().cpu().numpy() - want)
    assert np.all(err <= 16 * 2.0 ** -24 * size + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want))


def check_slots(e, k, v, slots):
    """What the cache holds there is k and v, quantised."""
    for x, codes, scales in ((k, e.cache.k_codes, e.cache.k_scales),
                             (v, e.cache.v_codes, e.cache.v_scales)):
        at = np.array(slots)
        ok = at >= 0
        if not ok.any():  # holes throughout
            continue
        c, s = kv4_reference.encode(x.double().cpu().numpy()[ok])
        want = kv4_reference.decode(kv4_reference.pack(c), s)
        got = kv4_reference.decode(codes.flatten(0, 1).cpu().numpy()[at[ok]],
                                   scales.flatten(0, 1).cpu().numpy()[at[ok]])
        assert np.array_equal(got, want)


@pytest.mark.parametrize("heads,group,dim,page", [(2, 4, 128, 16), (1, 7, 64, 4)])
def test_prompts_and_decoding_against_the_definitions(example, heads, group, dim, page):
    rows, limit = 5, 300
    lengths = [130, 1, 64, 0, 201]
    pages = sum(-(-n // page) for n in lengths) + 9  # the list runs out while decoding
    e = example.Engine(rows, limit, pages, page, heads, group, dim)
    model = Model(e, pages, page)
    gen = torch.Generator(device=DEV).manual_seed(heads)

    def projection(n):
        x = torch.randn(n, e.q_heads + 2 * heads, dim, generator=gen, device=DEV)
        return (1.5 * x).bfloat16()

    both = e.q_heads + heads
    places = sum(lengths) + 3  # the last ones stay empty
    fused = projection(places)
    before = fused.clone()
    fused[sum(lengths):] = float("nan")
    out, lse, step = e.prompts(fused, torch.tensor(lengths, dtype=torch.int32, device=DEV))
    want = model.place(lengths, places)
    assert [x.tolist() for x in step] == list(want[:7]) and e.table.tolist() == want[7]
    n = sum(lengths)
    check_turned(e, before[:n, :both], fused[:n, :both], want[1][:n])
    assert torch.equal(fused[:n, both:], before[:n, both:])
    q, k, v = fused.split([e.q_heads, heads, heads], 1)
    check_slots(e, k, v, want[0])
    w_out, w_lse, tol, lse_tol = ref.attention(q[:n], k[:n], v[:n], want[4])
    assert ((out[:n].double() - w_out).abs() <= tol + 2.0 ** -8 * (1 + 2.0 ** -8) * w_out.abs()
            ).all()
    assert ((lse[:n].double() - w_lse).abs() <= lse_tol).all()

    # decode steps from a graph, until the free pages are gone and beyond
    token = torch.empty(rows, e.q_heads + 2 * heads, dim, dtype=torch.bfloat16, device=DEV)
    token.copy_(projection(rows))
    e.decode(token)
    model.place([1] * rows, rows)
    graph = torch.cuda.CUDAGraph()
    token.copy_(projection(rows))
    with torch.cuda.graph(graph):
        out, lse, step = e.decode(token)
    for _ in range(3 * page):
        before = projection(rows)
        token.copy_(before)
        graph.replay()
        want = model.place([1] * rows, rows)
        assert [x.tolist() for x in step] == list(want[:7]) and e.table.tolist() == want[7]
        check_turned(e, before[:, :both], token[:, :both], want[1])
        q, k, v = token.split([e.q_heads, heads, heads], 1)
        check_slots(e, k, v, want[0])
        w_out, w_lse, _, tol, lse_tol, _ = kv4_reference.attention(
            model.planes(), q.double().cpu().numpy(), np.array(want[7]), want[3], owner=want[2])
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - w_out) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(w_out)
                      + 2.0 ** -25)
        assert np.all(np.abs(lse.double().cpu().numpy() - w_lse) <= lse_tol)
    assert model.used > pages and any(-1 in r[:-(-n // page)]
                                      for r, n in zip(model.table, model.lens))


def test_the_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["prompt_batch.py", "--rows", "4", "--prompt", "300",
                                      "--steps", "5"])
    example.main()
    said = capsys.readouterr().out
    assert "4 prompts" in said and "a decode step" in said

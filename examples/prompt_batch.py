"""Prompts and the decode steps that follow them, over a 4-bit cache.

What a serving engine does with each batch, with synthetic tensors in the model's
place: the new tokens get pages, slots and positions from the requests' lengths;
queries and keys are turned by their positions; keys and values enter the cache;
prompts attend over their own keys and values, single tokens over the cache.  The
decode step is captured in a CUDA graph: lengths, pages and the list of free
pages advance on the device, nothing is read back.

    python examples/prompt_batch.py --steps 64
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_stable_gb300 as dk  # noqa: E402


class Engine:
    """Up to `rows` sequences of up to `limit` tokens in a paged cache."""

    def __init__(self, rows, limit, pages, page_size=64, heads=8, group=8, dim=128, device="cuda"):
        self.rows, self.page_size, self.num_pages = rows, page_size, pages
        self.q_heads, self.heads = heads * group, heads
        self.cache = dk.Kv4Cache.allocate(pages, page_size, heads, dim, device)
        self.rope = dk.Rotary(dim, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((rows, -(-limit // page_size)), -1, **i32)
        self.lens = torch.zeros(rows, **i32)
        self.free = torch.arange(pages, **i32)
        self.used = torch.zeros(1, **i32)
        # a decode step's places, written anew by every replay
        self.one = torch.ones(rows, **i32)
        self.decode_step = dk.Kv4Step(
            torch.empty(rows, dtype=torch.int64, device=device),
            *[torch.empty(rows, **i32) for _ in range(3)],
            torch.empty(rows + 1, **i32), self.lens, self.used)

    def place(self, counts, places, out=None):
        """Pages, slots and positions for counts[b] new tokens of each sequence."""
        step = dk.kv4_extend(self.table, self.lens, counts, self.free, self.used, places,
                             self.page_size, self.num_pages, out=out)
        if out is None:
            self.lens.copy_(step.lens)
            self.used.copy_(step.used)
        return step

    def split(self, fused, step):
        """Queries, keys and values of a projection's output (places, q_heads + 2
        heads, dim): the first two turned in place, the others into the cache."""
        q, k, v = fused.split([self.q_heads, self.heads, self.heads], 1)
        dk.rotary(self.rope, step.positions, q, k, q_out=q, k_out=k)
        dk.kv4_append(self.cache, k, v, step.slots)
        return q, k, v

    def prompts(self, fused, counts):
        """New sequences' prompts, one after the other in fused; (out, lse, step)."""
        step = self.place(counts, len(fused))
        out, lse = dk.prompt_attention(*self.split(fused, step), step.starts)
        return out, lse, step

    def decode(self, fused):
        """One more token of every sequence; (out, lse, step)."""
        step = self.place(self.one, self.rows, out=self.decode_step)
        q, _, _ = self.split(fused, step)
        out, lse = dk.kv4_attention(self.cache, q, self.table, step.row_lens, owner=step.owner)
        return out, lse, step


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=2048, help="tokens of the longest prompt")
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    limit = a.prompt + a.steps + 8
    e = Engine(a.rows, limit, pages=a.rows * (-(-limit // 64)))
    gen = torch.Generator(device="cuda").manual_seed(0)

    def projection(tokens):
        x = torch.randn(tokens, e.q_heads + 2 * e.heads, e.cache.dim, generator=gen, device="cuda")
        return x.bfloat16()

    lengths = [a.prompt - i * a.prompt // (2 * a.rows) for i in range(a.rows)]
    counts = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    fused = projection(sum(lengths))
    e.prompts(fused[:1].clone(), torch.zeros_like(counts))  # loads the library
    torch.cuda.synchronize()
    t = time.perf_counter()
    e.prompts(fused, counts)
    torch.cuda.synchronize()
    print(f"{a.rows} prompts, {sum(lengths)} tokens: {1e6 * (time.perf_counter() - t):.0f} us")

    token = projection(a.rows)
    e.decode(token)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.decode(token)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        token.normal_(generator=gen)
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    print(f"{a.rows} sequences, up to {int(e.lens.max())} tokens: {1e6 * t:.0f} us a decode step, "
          f"{int(e.used)} of {e.num_pages} pages given away")


if __name__ == "__main__":
    main()

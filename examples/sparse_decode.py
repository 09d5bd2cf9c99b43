"""Sparse decoding over a 4-bit cache, one token of every sequence at a time.

What a serving engine does in each step, with synthetic tensors in the model's
place: the new tokens' keys and values enter the cache; the indexer's logits,
sharded over `dcp` ranks, give every row its top-K token ids; attention reads
only those tokens and accumulates their weights; a sequence that has outgrown
its budget is cut back to its heaviest tokens.

    python examples/sparse_decode.py --steps 64
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_stable_gb300 as dk  # noqa: E402


class Sequences:
    """`rows` sequences in a paged cache: each owns two runs of pages, the one it
    lives in and the one that an eviction copies into."""

    def __init__(self, rows, limit, page_size=64, heads=8, group=8, dim=128, dcp=4, top_k=512,
                 budget=1024, sinks=4, recent=128, device="cuda", seed=0):
        assert budget < limit and limit % (page_size * dcp) == 0
        self.rows, self.limit, self.dcp, self.top_k = rows, limit, dcp, top_k
        self.heads, self.group, self.dim = heads, group, dim
        self.budget, self.sinks, self.recent = budget, sinks, recent
        width = limit // page_size
        self.cache = dk.Kv4Cache.allocate(2 * rows * width, page_size, heads, dim, device)
        pages = torch.arange(2 * rows * width, dtype=torch.int32, device=device)
        self.table, self.spare = pages.view(2, rows, width).unbind(0)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=device)
        self.weights = torch.zeros(rows, limit, device=device)
        self.longest = 0  # on the host: all sequences grow together
        self.gen = torch.Generator(device=device).manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=self.lens.device)

    def append(self, k, v):
        """The next token of every sequence: k, v (rows, heads, dim)."""
        position = self.lens.long()
        size = self.cache.page_size
        page = self.table.long().gather(1, (position // size)[:, None])[:, 0]
        dk.kv4_append(self.cache, k, v, page * size + position % size)
        self.lens += 1
        self.longest += 1

    def select(self):
        """Every row's top-K ids by the indexer's logits, shard by shard."""
        shard = self.limit // self.dcp
        logits = self.normal(self.dcp, self.rows, shard)
        at = torch.arange(self.limit, device=logits.device).view(self.dcp, 1, shard)
        logits = logits.masked_fill(at >= self.lens[:, None], float("-inf"))
        return dk.fused_topk(logits, self.top_k)[1]

    def evict(self):
        kept, lens, weights = dk.kv4_evict(self.cache, self.table, self.lens, self.weights,
                                           self.spare, self.budget, sinks=self.sinks,
                                           recent=self.recent)
        self.table, self.spare = self.spare, self.table
        self.lens = lens
        self.weights.zero_()
        self.weights[:, :self.budget] = weights
        self.longest = min(self.longest, self.budget)
        return kept

    def step(self, k, v, q):
        """One decode step; returns (out, lse, the ids that were read)."""
        if self.longest == self.limit:
            self.evict()
        self.append(k, v)
        ids = self.select()
        out, lse = dk.kv4_attention(self.cache, q, self.table, self.lens, ids=ids,
                                    weights=self.weights, max_len=self.longest)
        return out, lse, ids

    def random_step(self):
        k, v = (self.normal(self.rows, self.heads, self.dim).bfloat16() for _ in range(2))
        q = 2 * self.normal(self.rows, self.heads * self.group, self.dim)
        return self.step(k, v, q.bfloat16())


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=16)
    ap.add_argument("--limit", type=int, default=2048, help="tokens before a sequence is cut back")
    ap.add_argument("--steps", type=int, default=256)
    a = ap.parse_args()
    s = Sequences(a.rows, a.limit)
    s.random_step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        s.random_step()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    print(f"{a.rows} sequences, {s.longest} tokens each after {a.steps + 1} steps: "
          f"{1e6 * t:.0f} us a step, the synthetic tensors included")


if __name__ == "__main__":
    main()

"""Attention over packed prompts, rotary positions and a batch's bookkeeping by
their definitions: 64 bits, exact angles, plain loops."""
from fractions import Fraction

import numpy as np

# 2 pi, to 50 digits
TURN = Fraction("6.28318530717958647692528676655900576839433879875021")


def attention(q, k, v, starts, *, causal=True, window=0, scale=None, softcap=0.0, p_step=2.0 ** -8):
    """(out, lse, bound on |out|'s error, bound on lse's error); torch tensors of
    64 bits.  Rows of no sequence stay NaN.

    The bounds are those of a kernel that sums exact products in fp32 and
    rounds probabilities to the type (p_step: half its step, relative):
    - a score: D + 8 roundings of 2^-24 of the sum of its products' magnitudes,
      the cap's tanh 2^-20 relative (of the cap at most), the exponent's
      argument 2^-22 of the score and of the maximum, exp2 2^-21;
    - the sum of the probabilities: 128 roundings of 2^-24 along the longest
      chain of a tile, and the tiles' sum compensated;
    - the second product: p_step, and n / 16 accumulations that may cut off a
      bit of 2^-23; fp16 probabilities below the smallest normal one are off by
      half a smallest step, 2^-25, where the largest is at least 2^4: 2^-29 each;
    - the output's rounding to its type is added by the caller."""
    import torch

    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64, device=q.device)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for a, b in zip(starts[:-1], starts[1:]):
        a, b = max(0, min(T, int(a))), max(0, min(T, int(b)))
        n = b - a
        if n <= 0:
            continue
        i = torch.arange(n, device=q.device)
        ok = torch.ones(n, n, dtype=torch.bool, device=q.device)
        if causal:
            ok &= i <= i[:, None]
        if window:
            ok &= i > i[:, None] - window
        for h in range(Hq):
            x0, kk, vv = q[a:b, h].double(), k[a:b, h // G].double(), v[a:b, h // G].double()
            x = torch.where(ok, x0 @ kk.T * scale, 0)
            dx = (D + 8) * 2.0 ** -24 * abs(scale) * torch.where(ok, x0.abs() @ kk.abs().T, 0)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                dx = torch.minimum(dx, dx * 0 + 2 * softcap) + 2.0 ** -20 * x.abs()
            top = torch.where(ok, x.abs(), 0).amax(-1, keepdim=True)
            dx = (dx + 2.0 ** -22 * (x.abs() + top)).amax(-1) + 2.0 ** -21
            x = torch.where(ok, x, -float("inf"))
            e = torch.logsumexp(x, -1)
            p = torch.exp(x - e[:, None])
            out[a:b, h] = p @ vv
            lse[a:b, h] = e
            seen = ok.sum(-1).double()
            sums = 128 * 2.0 ** -24
            rel = torch.expm1(2 * dx) + sums
            size = p @ vv.abs()
            tol[a:b, h] = size * (p_step * (1 + 2.0 ** -6) + rel + (seen / 16 + 32) * 2.0 ** -23
                                  )[:, None] + (seen * 2.0 ** -29)[:, None] * vv.abs().amax()
            lse_tol[a:b, h] = dx + sums + 2.0 ** -21 * (1 + e.abs())
    return out, lse, tol, lse_tol


def turned(x, positions, frequencies, *, interleaved=False, magnitude=1.0):
    """x (n, heads, D) float64 with its first 2 * len(frequencies) elements turned
    by exact angles."""
    half = len(frequencies)
    y = x.copy()
    for t, position in enumerate(positions):
        turns = [Fraction(f) * int(position) / TURN for f in frequencies]
        angle = np.array([float((a - round(a)) * TURN) for a in turns])
        c, s = np.cos(angle), np.sin(angle)
        first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
        second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
        a, b = x[t, :, first], x[t, :, second]
        y[t, :, first] = magnitude * (a * c - b * s)
        y[t, :, second] = magnitude * (b * c + a * s)
    return y


def extend(table, lens, counts, free, used, places, page_size, num_pages):
    """What kv4_extend returns, and the table after it; one token at a time."""
    table = [list(map(int, r)) for r in table]
    width = len(table[0]) if table else 0
    slots, positions, owner, row_lens, starts, out_lens = [], [], [], [], [], []
    used = max(0, int(used))
    for b, (held, count) in enumerate(zip(lens, counts)):
        held, count = max(0, int(held)), max(0, int(count))
        starts.append(len(slots))
        filled = -(-held // page_size)
        for _ in range(count):
            if len(slots) == places:
                break
            index = held // page_size
            if index < width and index >= filled:
                table[b][index] = int(free[used]) if used < len(free) else -1
                used += 1
                filled = index + 1
            page = table[b][index] if index < width else -1
            ok = 0 <= page < num_pages
            slots.append(page * page_size + held % page_size if ok else -1)
            positions.append(held)
            owner.append(b)
            held += 1
            row_lens.append(held)
        out_lens.append(held)
    starts.append(len(slots))
    pad = places - len(slots)
    return (slots + [-1] * pad, positions + [0] * pad, owner + [-1] * pad, row_lens + [0] * pad,
            starts, out_lens, [used], table)

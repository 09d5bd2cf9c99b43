"""The 4-bit key/value cache in 64 bits on the CPU, from its definition:
values of codes and scales, quantisation by distance to the grid, attention
row by row, eviction by sorting.  Nothing here is used by the library."""
from __future__ import annotations

import math

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_values():
    out = np.empty(127)
    for b in range(127):  # 127 is NaN
        e, m = b >> 3, b & 7
        out[b] = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return out


SCALES = _e4m3_values()


def nearest(x, grid):
    """Index of the nearest entry of an ascending grid for x >= 0: ties to the
    even index, beyond the last entry the last."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, x, side="left")   # x == mid stays below
    hi = np.searchsorted(mid, x, side="right")  # x == mid goes above
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


def encode(x, unit=1.0):
    """codes (..., D) as integers 0..15 and scales (..., D/16) as e4m3 bits."""
    x = np.asarray(x, np.float64) / unit
    x = x.reshape(*x.shape[:-1], -1, 16)
    a = np.where(np.isnan(x), 0.0, np.abs(x))
    bits = nearest(np.minimum(a.max(-1), 1e300) / 6.0, SCALES)
    s = SCALES[bits][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = nearest(np.where(s > 0, np.minimum(a, 1e300) / s, 0.0), MAGNITUDES)
    sign = np.where(np.isnan(x), 0, np.signbit(x)).astype(int)
    code = np.where(s > 0, code + 8 * sign, 0)
    return code.reshape(*code.shape[:-2], -1), bits


def pack(codes):
    codes = np.asarray(codes)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def decode(packed, scale_bits, unit=1.0):
    """Values (..., D) of packed codes (..., D/2) and scale bits (..., D/16)."""
    packed = np.asarray(packed)
    c = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1).astype(int)
    v = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.append(SCALES, np.nan)[np.asarray(scale_bits).astype(int) & 127]
    return v * np.repeat(s, 16, axis=-1) * unit


def row_positions(t, length, start, ids, row_start):
    """The positions that a row lists, in order (-1: none)."""
    length = max(0, int(length))
    start = max(0, int(start))
    if ids is None:
        return np.arange(start, max(start, length))
    out = []
    for i in ids[t]:
        p = int(i) - row_start
        out.append(p if i >= 0 and start <= p < length else -1)
    return np.array(out, int)


def attention(planes, q, table, lens, *, units=(1.0, 1.0), ids=None, owner=None, starts=None,
              row_starts=None, scale=None, softcap=0.0, positions=0):
    """(out, lse, weights, bound on |out|'s error, bound on lse's error) in
    64 bits.  planes: k_codes, v_codes, k_scales, v_scales as numpy arrays;
    q (T, Hq, D) float64.

    The bounds come from the kernel's roundings: products are exact and summed
    in fp32 (D + 4 roundings of at most 2^-24 of the sum of magnitudes, and
    the score's own scaling), exp and the running sum in fp32, probabilities
    rounded to fp16 (2^-11 of each, and 2^-25 at the least, where the largest
    is at least 1), the output rounded to its type (added by the caller)."""
    kc, vc, ks, vs = planes
    pages, page, H, _ = kc.shape
    T, Hq, D = q.shape
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    weights = np.zeros((T, positions))
    out_tol = np.zeros((T, Hq, D))
    lse_tol = np.zeros((T, Hq))
    w_tol = np.zeros((T, positions))
    for t in range(T):
        b = t if owner is None else int(owner[t])
        if not 0 <= b < table.shape[0]:
            continue
        length = min(int(lens[t]), table.shape[1] * page)
        pos = row_positions(t, length, 0 if starts is None else starts[t], ids,
                            0 if row_starts is None else int(row_starts[t]))
        pos = pos[pos >= 0]
        pg = table[b][pos // page]
        ok = (pg >= 0) & (pg < pages)
        pos, pg = pos[ok], pg[ok]
        if len(pos) == 0:
            continue
        off = pos % page
        K = decode(kc[pg, off], ks[pg, off], units[0])
        V = decode(vc[pg, off], vs[pg, off], units[1])
        n = len(pos)
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            x = k @ q[t, h] * scale
            dx = (D + 8) * 2.0 ** -24 * (np.abs(k) @ np.abs(q[t, h])) * abs(scale)
            if softcap:
                x = softcap * np.tanh(x / softcap)
                dx = dx + 2.0 ** -21 * softcap
            dx = (dx + 2.0 ** -22 * np.abs(x)).max() + 2.0 ** -21
            lse[t, h] = np.logaddexp.reduce(x)
            p = np.exp(x - lse[t, h])
            out[t, h] = p @ v
            size = p @ np.abs(v)
            sums = (n / 64 + 32) * 2.0 ** -24
            rel = np.expm1(2 * dx) + sums
            out_tol[t, h] = size * (2.0 ** -11 + rel) + n * 2.0 ** -25 * np.abs(v).max()
            lse_tol[t, h] = dx + sums + 2.0 ** -21 * (1 + abs(lse[t, h]))
            np.add.at(weights[t], pos[pos < positions], p[pos < positions])
            np.add.at(w_tol[t], pos[pos < positions], p[pos < positions] * (rel + 2.0 ** -20))
    return out, lse, weights, out_tol, lse_tol, w_tol


def evict(n, weights, budget, sinks, recent):
    """Kept positions, ascending."""
    if n <= budget:
        return np.arange(n)
    middle = list(range(sinks, n - recent))
    key = [-math.inf if math.isnan(weights[i]) else float(weights[i]) for i in range(n)]
    nan_last = [math.isnan(weights[i]) for i in range(n)]
    middle.sort(key=lambda i: (nan_last[i], -key[i], i))
    take = budget - sinks - recent
    return np.array(sorted(list(range(sinks)) + middle[:take] + list(range(n - recent, n))), int)

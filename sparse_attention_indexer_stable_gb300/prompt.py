"""What a batch's new tokens pass on their way into the 4-bit cache: tensor
conveniences over the C ABI of include/dcp_prompt.h.

``Rotary`` is a handle on the frequencies of rotary positions and ``rotary``
turns queries and keys by them; ``prompt_attention`` attends within whole
prompts over their own keys and values, before ``kv4_append`` quantises these.
As in the rest of the package all the work runs in the library's kernels on the
current CUDA stream (or on ``stream=``), nothing synchronises the host, and
there is no CPU fallback.
"""
from __future__ import annotations

import math
from fractions import Fraction

from . import _torch, kv4
from .kv4 import _handle, _raise

__all__ = ["Rotary", "rotary", "prompt_attention"]

_TURN = Fraction("6.2831853071795864769252867665590057683943")  # 2 pi


class Rotary:
    """The frequencies of rotary positions on one device.

    dim: how many elements of a head turn (its first ones), an even number;
    pair i of them turns by position * base ** (-2 i / dim) radians.
    interleaved: pair i is elements (2i, 2i + 1); otherwise (i, i + dim / 2).
    factor: for contexts `factor` times as long as the original one.  With
    original = 0 every frequency is divided by it.  With original, the length
    in tokens that the frequencies were made for, those that turn fewer than
    `slow` times over it are divided by the factor, those that turn more than
    `fast` times are kept, and between the two it is a linear blend.
    magnitude: multiplies the turned elements (default 1, with original
    0.1 ln(factor) + 1).
    frequencies: radians a position for each pair, in place of all of these (for
    checkpoints with another rule, such as a blend that is linear in the pair's
    index instead of its turns).
    Made once, outside of a CUDA graph's capture: exact fractions on the host, a
    tenth of a millisecond or two, and a copy to the device.
    """

    __slots__ = ("dim", "interleaved", "magnitude", "frequencies", "turns", "device")

    def __init__(self, dim, base=10000.0, interleaved=False, factor=1.0, original=0, slow=1.0,
                 fast=32.0, magnitude=None, frequencies=None, device="cuda"):
        torch = _torch()
        if dim < 2 or dim % 2 or dim > 1024:
            raise ValueError("dim must be even, between 2 and 1024")
        if frequencies is None:
            if not (math.isfinite(base) and base >= 1.0):
                raise ValueError("base must be finite and at least 1")
            if not (math.isfinite(factor) and factor >= 1.0):
                raise ValueError("factor must be finite and at least 1")
            if original < 0 or not 0.0 <= slow < fast:
                raise ValueError("need original >= 0 and 0 <= slow < fast")
            frequencies = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
            if factor != 1.0 and original:
                keep = [min(1.0, max(0.0, (original * f / (2.0 * math.pi) - slow) / (fast - slow)))
                        for f in frequencies]
                frequencies = [f * k + f / factor * (1.0 - k) for f, k in zip(frequencies, keep)]
                if magnitude is None:
                    magnitude = 0.1 * math.log(factor) + 1.0
            else:
                frequencies = [f / factor for f in frequencies]
        frequencies = [float(f) for f in frequencies]
        if len(frequencies) != dim // 2 or not all(math.isfinite(f) for f in frequencies):
            raise ValueError("frequencies must be dim / 2 finite numbers")
        magnitude = 1.0 if magnitude is None else float(magnitude)
        if not math.isfinite(magnitude):
            raise ValueError("magnitude must be finite")
        self.dim, self.interleaved, self.magnitude = int(dim), bool(interleaved), magnitude
        self.frequencies = tuple(frequencies)
        # 2^64 times the turns of a position, modulo 2^64, as int64
        turns = [round(Fraction(f) * 2 ** 64 / _TURN) % 2 ** 64 for f in frequencies]
        self.turns = torch.tensor([t - (t >> 63 << 64) for t in turns], dtype=torch.int64,
                                  device=device)
        if not self.turns.is_cuda:
            raise ValueError("device must be a CUDA device")
        self.device = self.turns.get_device()


def rotary(rope, positions, q, k=None, q_out=None, k_out=None, stream=None):
    """Turn the heads of q, and of k, by their tokens' positions: (q_out, k_out),
    k_out None without k.

    q: float16, bfloat16 or float32 (N, heads, D), any row and head strides; k:
    the same with its own number of heads; the elements of a head beyond
    rope.dim are copied.  positions: int32 (N,); a negative one turns back.
    q_out, k_out: contiguous new tensors by default; q_out=q (k_out=k) works in
    place, other overlaps do not.
    """
    if not isinstance(rope, Rotary):
        raise TypeError("rope must be a Rotary")
    r = (kv4._bound or kv4._bind()).rotary(rope.turns, rope.dim, rope.interleaved,
                                               rope.magnitude, positions, q, k, q_out, k_out,
                                               _handle(stream))
    if type(r) is int:
        _raise(r, "dcp_rotary")
    return r


def prompt_attention(q, k, v, starts, causal=True, window=0, scale=None, softcap=0.0, out=None,
                     lse=None, stream=None):
    """Attention within packed sequences: (out (T, q_heads, D) of q's dtype, lse
    float32 (T, q_heads), natural logarithm).

    q: float16 or bfloat16 (T, q_heads, D), D 64, 128 or 256; k, v: (T, heads, D)
    of q's dtype; query head h reads key/value head h // (q_heads // heads).  Any
    row and head strides; what is not 16-byte aligned, or whose strides are 0 or
    no multiples of 8 elements, is copied first.
    Products and sums are fp32; probabilities are rounded to q's dtype before they
    meet the values.  No gradients: inputs that require them are taken as they are.
    starts: int32 (sequences + 1,), ascending, as kv4_extend gives them: sequence
    b is rows starts[b] to starts[b + 1] - 1.  Row i of a sequence sees its rows
    j <= i (all of them with causal=False) and, with a window, j > i - window.
    scale: default (None or 0) D ** -0.5.  softcap: scores become
    softcap * tanh(score / softcap); 0: none.
    out, lse: contiguous; they share no memory with the inputs.  Rows of no sequence
    are left as they are in them; where they are allocated here, such rows hold no
    particular value.
    Largest scores beyond 2^20 ln 2, and infinities or NaN among values just
    behind what a row sees, are right but slow (some 200 times, for those rows).
    Should a copy not land within about a second, the rows that wait for it are NaN
    and dcp_topk_device_status() has DCP_DEVICE_COPY_TIMEOUT set.
    """
    r = (kv4._bound or kv4._bind()).prompt_attention(q, k, v, starts, causal, window, scale,
                                                     softcap, out, lse, _handle(stream))
    if type(r) is int:
        _raise(r, "dcp_prompt_attention")
    return r

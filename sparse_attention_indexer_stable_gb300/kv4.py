"""The 4-bit key/value cache beside the top-K: tensor conveniences over the C
ABI of include/dcp_kv4.h.

``Kv4Cache`` is a handle on four torch tensors (codes and scales of K and V in
pages); ``kv4_append`` and ``kv4_read`` write tokens and read them back,
``kv4_attention`` attends over every visible position of a row or over the ids
that ``merge`` and ``fused_topk`` give, ``kv4_evict`` keeps a sequence's
heaviest tokens.  As in the rest of the package all the work runs in the
library's kernels on the current CUDA stream (or on ``stream=``), nothing
synchronises the host, and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import struct
import threading

from . import DCP_OK, DcpError, _build, _check, _torch, library

__all__ = ["Kv4Cache", "kv4_append", "kv4_read", "kv4_attention", "kv4_attention_workspace_size",
           "kv4_evict", "DCP_F16", "DCP_BF16", "DCP_F32"]

DCP_F16, DCP_BF16, DCP_F32 = 0, 1, 2

# the C structs, native alignment
_CACHE = struct.Struct("PPPPqiiiff4x")
_ATTENTION = struct.Struct("PqqPqPPPPqPPqqPPPNiiiiiiiff4x")
_EVICT = struct.Struct("PqPPqPqPPPiiiiii")

_lock = threading.Lock()
_bound = None


def _bind():
    """The torch side of these functions (csrc/kv4_binding.cpp), connected to
    the library."""
    global _bound
    with _lock:
        if _bound is None:
            _torch()  # loads the libraries that the module is linked against
            lib = library()
            spec = importlib.util.spec_from_file_location("_kv4_binding", _build.build_binding())
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.connect(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.dcp_kv4_append, lib.dcp_kv4_read, lib.dcp_kv4_attention_workspace_size,
                lib.dcp_kv4_attention, lib.dcp_kv4_evict)])
            _bound = module
    return _bound


@functools.lru_cache(maxsize=None)
def _dtypes():
    torch = _torch()
    return {torch.float16: DCP_F16, torch.bfloat16: DCP_BF16, torch.float32: DCP_F32}


def _raise(status, where):
    if status != DCP_OK:
        raise DcpError(status, where)


def _handle(stream):
    """A raw stream handle, or None for the current stream."""
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Kv4Cache:
    """A handle on a paged cache of 4-bit keys and values.

    k_codes, v_codes: uint8 (pages, page_size, heads, dim / 2); k_scales,
    v_scales: uint8 (pages, page_size, heads, dim / 16), e4m3 bits; all
    contiguous CUDA tensors of one device.  dim is 64, 128 or 256, page_size a
    power of two.  An element stands for unit * scale * e2m1(code); k_unit and
    v_unit are powers of two that bring the values of K and V into the scales'
    range (a block's largest magnitude between about 0.01 and 2688 units).
    """

    __slots__ = ("k_codes", "v_codes", "k_scales", "v_scales", "num_pages", "page_size", "heads",
                 "dim", "k_unit", "v_unit", "device", "_raw")

    def __init__(self, k_codes, v_codes, k_scales, v_scales, k_unit=1.0, v_unit=1.0):
        torch = _torch()
        _check(k_codes, "k_codes", torch.uint8, None)
        dev = k_codes.get_device()
        for name, t in (("v_codes", v_codes), ("k_scales", k_scales), ("v_scales", v_scales)):
            _check(t, name, torch.uint8, dev)
        if k_codes.dim() != 4 or v_codes.shape != k_codes.shape:
            raise ValueError("k_codes and v_codes must both be (pages, page_size, heads, dim / 2)")
        pages, page_size, heads, half = k_codes.shape
        scales = (pages, page_size, heads, half // 8)
        if half % 8 or k_scales.shape != scales or v_scales.shape != scales:
            raise ValueError("k_scales and v_scales must both be (pages, page_size, heads, dim / 16)")
        self.k_codes, self.v_codes = k_codes, v_codes
        self.k_scales, self.v_scales = k_scales, v_scales
        self.num_pages, self.page_size, self.heads, self.dim = pages, page_size, heads, 2 * half
        self.k_unit, self.v_unit = float(k_unit), float(v_unit)
        self.device = dev
        self._raw = _CACHE.pack(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                v_scales.data_ptr(), pages, page_size, heads, self.dim,
                                self.k_unit, self.v_unit)
        # an empty append checks the sizes, the units and the alignment
        _raise(library().dcp_kv4_append(self._raw, None, None, DCP_BF16, 0, 0, 0, 0, 0, None,
                                        None), "Kv4Cache")

    @classmethod
    def allocate(cls, num_pages, page_size, heads, dim, device="cuda", k_unit=1.0, v_unit=1.0):
        """A cache of zeros on `device`."""
        torch = _torch()
        if dim % 16:
            raise ValueError("dim must be 64, 128 or 256")
        planes = [torch.zeros((num_pages, page_size, heads, w), dtype=torch.uint8, device=device)
                  for w in (dim // 2, dim // 2, dim // 16, dim // 16)]
        return cls(*planes, k_unit=k_unit, v_unit=v_unit)


def _cache(cache):
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")


def kv4_append(cache, k, v, slots, stream=None):
    """Quantise N tokens and write them to their slots.

    k, v: (N, heads, dim) of float16, bfloat16 or float32, any row and head
    strides; slots: int64 (N,), page * page_size + offset; tokens whose slot is
    outside the cache (for example -1) are skipped.  Slots are distinct.
    """
    _cache(cache)
    _raise((_bound or _bind()).append(cache._raw, cache.device, k, v, slots, _handle(stream)),
           "dcp_kv4_append")


def kv4_read(cache, slots, dtype=None, k=None, v=None, stream=None):
    """What the slots stand for: (k, v), each (N, heads, dim) of dtype
    (default bfloat16).  Slots outside the cache read as zeros.
    """
    _cache(cache)
    if dtype is None:
        dtype = _torch().bfloat16 if k is None else k.dtype
    if dtype not in _dtypes():
        raise TypeError("dtype must be float16, bfloat16 or float32")
    r = (_bound or _bind()).read(cache._raw, cache.device, slots, _dtypes()[dtype], k, v,
                                 _handle(stream))
    if type(r) is int:
        _raise(r, "dcp_kv4_read")
    return r


def kv4_attention_workspace_size(cache, rows, q_heads, table_width, num_ids=None, max_len=0,
                                 weights=False):
    """Workspace bytes of kv4_attention for these sizes (num_ids: None without
    ids); table_width is the block table's pages per sequence."""
    _cache(cache)
    args = _ATTENTION.pack(0, 0, 0, 0, 0, 0, 0, 0, 0 if num_ids is None else 16, 0, 0,
                           16 if weights else 0, 0, 0, 0, 0, 0, 0, DCP_BF16, rows, q_heads, rows,
                           table_width, num_ids or 0, max_len, 0.0, 0.0)
    n = ctypes.c_size_t(0)
    _raise(library().dcp_kv4_attention_workspace_size(cache._raw, args, ctypes.byref(n)),
           "dcp_kv4_attention_workspace_size")
    return n.value


def kv4_attention(cache, q, table, lens, ids=None, owner=None, starts=None, row_starts=None,
                  scale=None, softcap=0.0, weights=None, max_len=0, out=None, lse=None,
                  workspace=None, stream=None):
    """Attention of T query rows over the cache: (out (T, q_heads, dim) of q's
    dtype, lse float32 (T, q_heads), natural logarithm).

    q: float16 or bfloat16 (T, q_heads, dim), any row and head strides; query
    head h reads key/value head h // (q_heads // heads).
    table: int32 (sequences, pages per sequence), the block table; entries
    outside the cache are holes, whose tokens are absent.
    lens, starts: int32 (T,); row t sees positions starts[t] <= p < lens[t]
    (starts: default 0).  owner: int32 (T,), the rows' sequences (default: row
    t is sequence t).
    ids: int32 (T, K), as merge and fused_topk return them: the row attends
    only to these positions (those that it sees); -1 is padding.  row_starts:
    int32 (T,), subtracted from the ids, as it was added by the top-K.
    scale: default (None or 0) dim ** -0.5.  softcap: scores become
    softcap * tanh(score / softcap); 0: none.
    weights: float32 (T, positions), unit column stride: each position's
    probability, summed over the query heads, is added (not with owner).
    max_len: a host-side bound of lens (0: the table's width); the launch is
    shaped by it, and positions from it on are not seen.
    A row that sees nothing gives zeros and lse -inf.
    """
    _cache(cache)
    r = (_bound or _bind()).attention(cache._raw, cache.device, q, table, lens, ids, owner, starts,
                                      row_starts, scale, softcap, weights, max_len, out, lse,
                                      workspace, _handle(stream))
    if type(r) is int:
        _raise(r, "dcp_kv4_attention")
    return r


def kv4_evict(cache, table, lens, weights, out_table, budget, sinks=0, recent=0, kept=None,
              out_lens=None, out_weights=None, stream=None):
    """Copy the tokens worth keeping into other pages of the cache.

    table: int32 (sequences, pages); lens: int32 (sequences,); weights: float32
    (sequences, positions), unit column stride, as kv4_attention accumulates
    them; out_table: int32 (sequences, at least ceil(budget / page_size)), pages
    that are in no row of table.  A sequence of at most budget tokens keeps
    them all; a longer one keeps its first `sinks`, its last `recent` and the
    heaviest of the others (equal weights: the lowest position), in order; a
    kept token on a hole of table becomes zeros.
    Returns (kept int32 (sequences, budget): the kept positions, ascending, then
    -1; out_lens int32; out_weights float32 (sequences, budget)).
    """
    _cache(cache)
    r = (_bound or _bind()).evict(cache._raw, cache.device, table, lens, weights, out_table,
                                  budget, sinks, recent, kept, out_lens, out_weights,
                                  _handle(stream))
    if type(r) is int:
        _raise(r, "dcp_kv4_evict")
    return r

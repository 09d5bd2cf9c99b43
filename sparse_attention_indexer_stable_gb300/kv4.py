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

import functools
import struct

from . import DCP_OK, DcpError, _check, _on_device, _stream_handle, _torch, library

__all__ = ["Kv4Cache", "kv4_append", "kv4_read", "kv4_attention", "kv4_attention_workspace_size",
           "kv4_evict", "DCP_F16", "DCP_BF16", "DCP_F32"]

DCP_F16, DCP_BF16, DCP_F32 = 0, 1, 2

# the C structs, native alignment
_CACHE = struct.Struct("PPPPqiiiff4x")
_ATTENTION = struct.Struct("PqqPqPPPPqPPqqPPPNiiiiiiiff4x")
_EVICT = struct.Struct("PqPPqPqPPPiiiiii")


@functools.lru_cache(maxsize=None)
def _dtypes():
    torch = _torch()
    return {torch.float16: DCP_F16, torch.bfloat16: DCP_BF16, torch.float32: DCP_F32}


def _raise(status, where):
    if status != DCP_OK:
        raise DcpError(status, where)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _allocating(stream, dev):
    """A context in which torch allocates for `stream`: what a call allocates
    may then be freed as soon as the call returns."""
    torch = _torch()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_handle(stream, dev), device=dev)
    return torch.cuda.stream(stream)


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
                 "dim", "k_unit", "v_unit", "device", "_raw", "_key")

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
        self._key = (pages, page_size, heads, self.dim)
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


def _rows(t, name, dtype, dev, what):
    """A 2-D tensor whose rows are contiguous (at any stride)."""
    if not isinstance(t, _torch().Tensor) or t.dtype != dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on cuda:{dev}")
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1 and t.shape[0]):
        raise ValueError(f"{name} must be {what}, its rows contiguous")


def _cache(cache):
    if not isinstance(cache, Kv4Cache):
        raise TypeError("cache must be a Kv4Cache")
    return cache.device


def _values(t, name, cache, dtypes):
    """(n, heads, dim) values with unit stride along dim, on the cache's device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{name} must be a torch.Tensor of float16, bfloat16"
                        + (" or float32" if len(dtypes) > 2 else ""))
    if t.get_device() != cache.device:
        raise ValueError(f"{name} must be on cuda:{cache.device}")
    if t.dim() != 3 or t.shape[2] != cache.dim or t.stride(2) != 1:
        raise ValueError(f"{name} must be 3-D, its last dimension dim = {cache.dim} contiguous")


def kv4_append(cache, k, v, slots, stream=None):
    """Quantise N tokens and write them to their slots.

    k, v: (N, heads, dim) of float16, bfloat16 or float32, any row and head
    strides; slots: int64 (N,), page * page_size + offset; tokens whose slot is
    outside the cache (for example -1) are skipped.  Slots are distinct.
    """
    dev = _cache(cache)
    _values(k, "k", cache, _dtypes())
    _values(v, "v", cache, _dtypes())
    if k.dtype != v.dtype or k.shape != v.shape or k.shape[1] != cache.heads:
        raise ValueError("k and v must both be (N, heads, dim) of one dtype")
    _check(slots, "slots", _torch().int64, dev)
    if slots.shape != (k.shape[0],):
        raise ValueError("slots must be (N,)")
    kr, kh, _ = k.stride()
    vr, vh, _ = v.stride()
    _raise(_on_device(dev, lambda: library().dcp_kv4_append(
        cache._raw, k.data_ptr(), v.data_ptr(), _dtypes()[k.dtype], k.shape[0], kr, kh, vr, vh,
        slots.data_ptr(), _stream_handle(stream, dev))), "dcp_kv4_append")


def kv4_read(cache, slots, dtype=None, k=None, v=None, stream=None):
    """What the slots stand for: (k, v), each (N, heads, dim) of dtype
    (default bfloat16).  Slots outside the cache read as zeros.
    """
    torch = _torch()
    dev = _cache(cache)
    _check(slots, "slots", torch.int64, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be (N,)")
    if dtype is None:
        dtype = k.dtype if k is not None else torch.bfloat16
    if dtype not in _dtypes():
        raise TypeError("dtype must be float16, bfloat16 or float32")
    shape = (slots.shape[0], cache.heads, cache.dim)
    if k is None or v is None:
        if stream is None:
            k = torch.empty(shape, dtype=dtype, device=dev) if k is None else k
            v = torch.empty(shape, dtype=dtype, device=dev) if v is None else v
        else:
            with _allocating(stream, dev):
                k = torch.empty(shape, dtype=dtype, device=dev) if k is None else k
                v = torch.empty(shape, dtype=dtype, device=dev) if v is None else v
    _check(k, "k", dtype, dev)
    _check(v, "v", dtype, dev)
    if k.shape != shape or v.shape != shape:
        raise ValueError("k and v must be (N, heads, dim)")
    _raise(_on_device(dev, lambda: library().dcp_kv4_read(
        cache._raw, k.data_ptr(), v.data_ptr(), _dtypes()[dtype], shape[0], slots.data_ptr(),
        _stream_handle(stream, dev))), "dcp_kv4_read")
    return k, v


@functools.lru_cache(maxsize=1024)
def _workspace_size(key, rows, q_heads, num_seqs, table_width, num_ids, max_len, weights):
    import ctypes

    pages, page_size, heads, dim = key
    raw = _CACHE.pack(16, 16, 16, 16, pages, page_size, heads, dim, 1.0, 1.0)
    ids = 0 if num_ids is None else 16
    args = _ATTENTION.pack(0, 0, 0, 0, 0, 0, 0, 0, ids, 0, 0, 16 if weights else 0, 0, 0, 0, 0, 0,
                           0, DCP_BF16, rows, q_heads, num_seqs, table_width, num_ids or 0,
                           max_len, 0.0, 0.0)
    n = ctypes.c_size_t(0)
    _raise(library().dcp_kv4_attention_workspace_size(raw, args, ctypes.byref(n)),
           "dcp_kv4_attention_workspace_size")
    return n.value


def kv4_attention_workspace_size(cache, rows, q_heads, table_width, num_ids=None, max_len=0,
                                 weights=False):
    """Workspace bytes of kv4_attention for these sizes (num_ids: None without
    ids); table_width is the block table's pages per sequence."""
    _cache(cache)
    return _workspace_size(cache._key, rows, q_heads, rows, table_width, num_ids, max_len,
                           bool(weights))


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
    scale: default dim ** -0.5.  softcap: scores become
    softcap * tanh(score / softcap); 0: none.
    weights: float32 (T, positions), unit column stride: each position's
    probability, summed over the query heads, is added (not with owner).
    max_len: a host-side bound of lens (0: the table's width); it only shapes
    the launch, and lens beyond it are cut there.
    A row that sees nothing gives zeros and lse -inf.
    """
    torch = _torch()
    dev = _cache(cache)
    dtypes = _dtypes()
    if isinstance(q, torch.Tensor) and q.dtype == torch.float32:
        raise TypeError("q must be a torch.Tensor of float16, bfloat16")
    _values(q, "q", cache, dtypes)
    T, heads, dim = q.shape
    if heads < 1 or heads % cache.heads:
        raise ValueError("q's heads must be a multiple of the cache's heads")
    int32 = torch.int32
    _rows(table, "table", int32, dev, "(sequences, pages)")
    _check(lens, "lens", int32, dev)
    if lens.shape != (T,):
        raise ValueError("lens must be (T,)")
    for name, t in (("starts", starts), ("owner", owner), ("row_starts", row_starts)):
        if t is not None:
            _check(t, name, int32, dev)
            if t.shape != (T,):
                raise ValueError(f"{name} must be (T,)")
    num_seqs, width = table.shape
    if owner is None and num_seqs < T:
        raise ValueError("table must have a row for each row of q (or give owner)")
    num_ids, ids_ptr, ids_stride = None, 0, 0
    if ids is not None:
        _rows(ids, "ids", int32, dev, "(T, K)")
        if ids.shape[0] != T:
            raise ValueError("ids must be (T, K)")
        num_ids, ids_stride = ids.shape[1], ids.stride(0)
        # no ids at all (K = 0) have no address, and a null one means every
        # position; nothing is read from this one
        ids_ptr = ids.data_ptr() or lens.data_ptr()
    w_stride = w_width = 0
    if weights is not None:
        _rows(weights, "weights", torch.float32, dev, "(T, positions)")
        if owner is not None:
            raise ValueError("weights need one row per sequence: not with owner")
        if weights.shape[0] != T:
            raise ValueError("weights must be (T, positions)")
        w_stride, w_width = weights.stride(0), weights.shape[1]
        if T > 1 and w_stride < w_width:
            raise ValueError("the rows of weights must not overlap")
    if not softcap >= 0.0:
        raise ValueError("softcap must not be negative")
    need = _workspace_size(cache._key, T, heads, num_seqs, width, num_ids, max_len,
                           weights is not None)
    if out is None or lse is None or (need and workspace is None):
        if stream is None:
            out, lse, workspace = _outputs(torch, q, T, heads, dim, dev, need, out, lse,
                                           workspace)
        else:
            with _allocating(stream, dev):
                out, lse, workspace = _outputs(torch, q, T, heads, dim, dev, need, out, lse,
                                               workspace)
    _check(out, "out", q.dtype, dev)
    _check(lse, "lse", torch.float32, dev)
    if out.shape != (T, heads, dim) or lse.shape != (T, heads):
        raise ValueError("out must be (T, q_heads, dim) and lse (T, q_heads)")
    have = 0
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, dev)
        have = workspace.numel()
        if have < need:
            raise ValueError(f"workspace must hold {need} bytes")
    args = _ATTENTION.pack(
        q.data_ptr(), q.stride(0), q.stride(1), table.data_ptr(), table.stride(0),
        lens.data_ptr(), _ptr(starts), _ptr(owner), ids_ptr, ids_stride, _ptr(row_starts),
        _ptr(weights), w_stride, w_width, out.data_ptr(), lse.data_ptr(), _ptr(workspace), have,
        dtypes[q.dtype], T, heads, num_seqs, width, num_ids or 0, max_len, scale or 0.0, softcap)
    _raise(_on_device(dev, lambda: library().dcp_kv4_attention(
        cache._raw, args, _stream_handle(stream, dev))), "dcp_kv4_attention")
    return out, lse


def _outputs(torch, q, T, heads, dim, dev, need, out, lse, workspace):
    if out is None:
        out = torch.empty((T, heads, dim), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((T, heads), dtype=torch.float32, device=dev)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return out, lse, workspace


def kv4_evict(cache, table, lens, weights, out_table, budget, sinks=0, recent=0, kept=None,
              out_lens=None, out_weights=None, stream=None):
    """Copy the tokens worth keeping into other pages of the cache.

    table: int32 (sequences, pages); lens: int32 (sequences,); weights: float32
    (sequences, positions), unit column stride, as kv4_attention accumulates
    them; out_table: int32 (sequences, at least ceil(budget / page_size)), pages
    that are in no row of table.  A sequence of at most budget tokens keeps
    them all; a longer one keeps its first `sinks`, its last `recent` and the
    heaviest of the others (equal weights: the lowest position), in order.
    Returns (kept int32 (sequences, budget): the kept positions, ascending, then
    -1; out_lens int32; out_weights float32 (sequences, budget)).
    """
    torch = _torch()
    dev = _cache(cache)
    int32 = torch.int32
    budget, sinks, recent = int(budget), int(sinks), int(recent)
    if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("need budget >= 1, sinks >= 0, recent >= 0, sinks + recent <= budget")
    _rows(table, "table", int32, dev, "(sequences, pages)")
    _rows(out_table, "out_table", int32, dev, "(sequences, pages)")
    _rows(weights, "weights", torch.float32, dev, "(sequences, positions)")
    B, width = table.shape
    if weights.shape[0] != B or out_table.shape[0] != B:
        raise ValueError("table, weights and out_table must have a row for each sequence")
    if out_table.shape[1] * cache.page_size < budget:
        raise ValueError("out_table must have ceil(budget / page_size) pages for each sequence")
    _check(lens, "lens", int32, dev)
    if lens.shape != (B,):
        raise ValueError("lens must have an entry for each sequence")
    if kept is None or out_lens is None or out_weights is None:
        if stream is None:
            kept, out_lens, out_weights = _kept(torch, B, budget, dev, kept, out_lens,
                                                out_weights)
        else:
            with _allocating(stream, dev):
                kept, out_lens, out_weights = _kept(torch, B, budget, dev, kept, out_lens,
                                                    out_weights)
    _check(kept, "kept", int32, dev)
    _check(out_lens, "out_lens", int32, dev)
    _check(out_weights, "out_weights", torch.float32, dev)
    if (kept.shape != (B, budget) or out_weights.shape != (B, budget)
            or out_lens.shape != (B,)):
        raise ValueError("kept and out_weights must be (sequences, budget), out_lens (sequences,)")
    args = _EVICT.pack(table.data_ptr(), table.stride(0), lens.data_ptr(), weights.data_ptr(),
                       weights.stride(0), out_table.data_ptr(), out_table.stride(0),
                       kept.data_ptr(), out_lens.data_ptr(), out_weights.data_ptr(), B, width,
                       weights.shape[1], budget, sinks, recent)
    _raise(_on_device(dev, lambda: library().dcp_kv4_evict(
        cache._raw, args, _stream_handle(stream, dev))), "dcp_kv4_evict")
    return kept, out_lens, out_weights


def _kept(torch, B, budget, dev, kept, out_lens, out_weights):
    if kept is None:
        kept = torch.empty((B, budget), dtype=torch.int32, device=dev)
    if out_lens is None:
        out_lens = torch.empty((B,), dtype=torch.int32, device=dev)
    if out_weights is None:
        out_weights = torch.empty((B, budget), dtype=torch.float32, device=dev)
    return kept, out_lens, out_weights

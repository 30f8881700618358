"""A serving step around the 4-bit key/value cache: pages for new tokens, and
norms, rotation and the cache write in one pass.

Thin binding over the C ABI in ``include/int4dq_cache_step.h`` (part of
``libint4dq.so``), in the manner of ``dequantizing_gemm_amd.cache``. A step of
a batch whose plan stays on the GPU:

    lengths, count = int4_cache_release(page_table, lengths, free, count, page_size, done)
    lengths, starts, slots, count = int4_cache_extend(page_table, lengths, free, count, page_size, new, rows=rows)
    q = int4_cache_append(cache, q, k, v, page_table, lengths, starts, q_norm=..., k_norm=..., rope=...)
    out = int4_cache_attention(q, cache, page_table, lengths, starts)

``free`` int32 [pages] holds the numbers of the free pages in its first
``count[0]`` entries; ``count`` int32 [2] also says how many pages the last
int4_cache_extend lacked. Both calls give new lengths and counts and leave the
ones they were given as they were, unless these are passed as ``out``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _gpu, _raise, lib
from .cache import (ROWS_DTYPES, Int4Cache, _call, _int32, _is_cache, _plan, _raw_stream, _rows_array)

__all__ = ["int4_cache_release", "int4_cache_extend", "int4_cache_append"]

_i64, _vp, _int = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int


class _PoolStruct(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("table_stride", _i64), ("max_pages", _i64), ("batch", _i64), ("page_size", _i64),
                ("free", _vp), ("pages", _i64)]


class _TransformStruct(ctypes.Structure):
    _fields_ = [("q_norm", _vp), ("k_norm", _vp), ("eps", ctypes.c_double), ("rope", _vp), ("rope_stride", _i64),
                ("rope_positions", _i64), ("rotary_dim", _i64), ("interleaved", _int)]


# Every function declared in include/int4dq_cache_step.h, with its ctypes signature.
CACHE_STEP_SIGNATURES = {
    "int4_cache_release": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "int4_cache_extend": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "int4_cache_append": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _int, _vp, _vp]),
    "int4_cache_attention_ex": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _i64, ctypes.c_float, _int, _i64, _i64, _vp, _i64,
                                       _vp, _vp, _vp, _i64, _vp]),
    "int4_cache_attention_ex_workspace_bytes": (_i64, [_vp, _vp, _i64, _int, _i64]),
}
for _name, (_res, _args) in CACHE_STEP_SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


def _flat(name, t, dtype, size, device):
    """A contiguous GPU vector of `size` elements, on `device` where that is given."""
    _gpu(t, name, dtype, 1)
    if size is not None and t.shape[0] != size:
        raise ValueError(f"{name} must have {size} entries (got {t.shape[0]})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    return t.data_ptr()


def _pool(page_table, lengths, free, count, page_size):
    """The pool descriptor, checked."""
    _flat("free", free, torch.int32, None, None)
    dev = free.device
    if not isinstance(page_table, torch.Tensor) or page_table.dtype != torch.int32 or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 tensor of 2 dimension(s)")
    if page_table.device != dev:
        raise ValueError(f"page_table must be on {dev} (got {page_table.device})")
    batch, max_pages = page_table.shape
    if page_table.numel() and max_pages > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table must be contiguous in its last dimension")
    stride = page_table.stride(0) if batch > 1 else max_pages
    if stride < max_pages:
        raise ValueError("page_table rows must not overlap")
    _flat("lengths", lengths, torch.int32, batch, dev)
    _flat("count", count, torch.int32, 2, dev)
    return _PoolStruct(page_table.data_ptr(), stride, max_pages, batch, page_size, free.data_ptr(), free.shape[0])


def _pool_call(fn, what, device, pool, *args):
    """Calls a C entry point with `device` current, on its current stream."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = fn(ctypes.addressof(pool), *args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(ctypes.addressof(pool), *args, _raw_stream(index))
    if rc:
        _raise(rc, what)


def int4_cache_release(page_table: torch.Tensor, lengths: torch.Tensor, free: torch.Tensor, count: torch.Tensor,
                       page_size: int, done: torch.Tensor, *, shared: torch.Tensor | None = None,
                       out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Give the pages of the sequences with ``done`` (bool or uint8 [batch]) back to
    ``free``; ``page_table`` is not changed. Returns (lengths, count): the lengths,
    0 for those sequences, and the free pages. ``shared`` int32 [1]: the pages
    wholly in the first shared[0] tokens belong to other sequences too and are kept.
    ``out``: the two tensors to fill, which may be ``lengths`` and ``count``."""
    pool = _pool(page_table, lengths, free, count, page_size)
    dev, batch = free.device, page_table.shape[0]
    if not isinstance(done, torch.Tensor) or done.dtype not in (torch.bool, torch.uint8):
        raise ValueError("done must be a bool or uint8 tensor")
    ended = _flat("done", done, done.dtype, batch, dev)
    common = None if shared is None else _flat("shared", shared, torch.int32, 1, dev)
    if out is None:
        out = (torch.empty(batch, dtype=torch.int32, device=dev), torch.empty(2, dtype=torch.int32, device=dev))
    to = [_flat(n, t, torch.int32, s, dev) for n, t, s in zip(("out[0]", "out[1]"), out, (batch, 2))]
    _pool_call(lib.int4_cache_release, "int4_cache_release", dev, pool, lengths.data_ptr(), ended, count.data_ptr(), common,
               *to)
    return out


def int4_cache_extend(page_table: torch.Tensor, lengths: torch.Tensor, free: torch.Tensor, count: torch.Tensor,
                      page_size: int, new: torch.Tensor | None = None, *, rows: int | None = None, slots: bool = True,
                      out: tuple | None = None):
    """Pages for ``new`` tokens (int32 [batch]; default one each) of each sequence, from
    ``free`` into ``page_table``, where these are enough; -1 where not. Returns (lengths,
    starts, slots, count): the lengths with the new tokens; the row offsets of the
    packed new tokens, int32 [batch + 1]; for each of ``rows`` rows (the sum of ``new``
    or more, known to the caller) the slot page * page_size + offset of its token, int64,
    -1 where it has none (None with ``slots=False``); and the free pages with how many
    more were needed. ``out``: the four to fill, of which the first and last may be
    ``lengths`` and ``count``."""
    pool = _pool(page_table, lengths, free, count, page_size)
    dev, batch = free.device, page_table.shape[0]
    added = None if new is None else _flat("new", new, torch.int32, batch, dev)
    if rows is None:
        if slots and new is not None and out is None:
            raise ValueError("rows must be given with new")
        rows = batch if new is None else out[2].shape[0] if out is not None and out[2] is not None else 0
    if out is None:
        def make(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=dev)
        out = (make(batch), make(batch + 1), make(rows, torch.int64) if slots else None, make(2))
    at = None if out[2] is None else _flat("out[2]", out[2], torch.int64, rows, dev)
    to = [_flat(f"out[{i}]", out[i], torch.int32, s, dev) for i, s in ((0, batch), (1, batch + 1), (3, 2))]
    _pool_call(lib.int4_cache_extend, "int4_cache_extend", dev, pool, lengths.data_ptr(), added, count.data_ptr(), to[0],
               to[1], at, rows, to[2])
    return out


def int4_cache_append(cache: Int4Cache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                      lengths: torch.Tensor, starts: torch.Tensor | None = None, *, q_norm: torch.Tensor | None = None,
                      k_norm: torch.Tensor | None = None, eps: float = 1e-6, rope: torch.Tensor | None = None,
                      interleaved: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """One pass from a projection's output to attention: q [rows, q_heads, head_dim]
    normalised for each head and rotated (returned, of its type), k and v [rows,
    heads, head_dim] quantised into the cache at the rows' positions, k normalised
    and rotated before. All three float32, float16 or bfloat16, any row and head strides.

    ``q_norm``, ``k_norm`` float32 [head_dim]: weights of x / sqrt(mean(x^2) + eps);
    None: no norm. ``rope`` float32 [positions, rotary_dim]: cosines, then sines, of
    the angles at each position; the first rotary_dim channels are rotated, in halves
    (i, i + rotary_dim / 2) or ``interleaved`` (2 i, 2 i + 1); None: no rotation. A row
    whose position is below 0 or past ``rope`` gives 0 and writes nothing. ``out``: a
    contiguous tensor to fill, which may be ``q``."""
    _is_cache(cache)
    q_heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
    qs = _rows_array(cache, q, "q", q_heads)
    ks, vs = _rows_array(cache, k, "k", cache.heads), _rows_array(cache, v, "v", cache.heads)
    if q.dtype not in ROWS_DTYPES or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError(f"q, k and v must be float32, float16 or bfloat16, all the same (got {q.dtype}, {k.dtype}, {v.dtype})")
    rows = q.shape[0]
    if k.shape[0] != rows or v.shape[0] != rows:
        raise ValueError(f"q has {rows} rows, k {k.shape[0]}, v {v.shape[0]}")
    plan = _plan(cache, page_table, lengths, starts, rows)
    weights = [None if w is None else _flat(n, w, torch.float32, cache.head_dim, cache.device)
               for n, w in (("q_norm", q_norm), ("k_norm", k_norm))]
    turn = (None, 0, 0, 0)
    if rope is not None:
        if not isinstance(rope, torch.Tensor) or rope.dtype != torch.float32 or rope.dim() != 2:
            raise ValueError("rope must be a float32 tensor of 2 dimensions")
        if rope.device != cache.device:
            raise ValueError(f"rope must be on {cache.device} (got {rope.device})")
        if rope.shape[1] > 1 and rope.stride(1) != 1:
            raise ValueError("rope must be contiguous in its last dimension")
        turn = (rope.data_ptr(), rope.stride(0) if rope.shape[0] > 1 else rope.shape[1], rope.shape[0], rope.shape[1])
    transform = _TransformStruct(*weights, eps, *turn, bool(interleaved))
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _gpu(out, "out", q.dtype, 3)
        if tuple(out.shape) != tuple(q.shape) or out.device != q.device:
            raise ValueError(f"out must be {tuple(q.shape)} on {q.device}")
    _call(cache, lib.int4_cache_append, "int4_cache_append", ctypes.addressof(plan), ctypes.addressof(transform),
          q.data_ptr(), *qs, q_heads, k.data_ptr(), *ks, v.data_ptr(), *vs, ROWS_DTYPES[q.dtype], out.data_ptr())
    return out

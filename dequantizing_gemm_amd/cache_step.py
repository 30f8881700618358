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
from .cache import ROWS_DTYPES, Int4Cache, _is_cache, _raw_stream, _rows_array, _RowsStruct

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


_Tensor, _int32_type = torch.Tensor, torch.int32

# A step's calls are short (5 us on the GPU): checks are put as one expression each, and
# what fails it goes through the checks that say what is wrong.


def _vector(t, name, dtype, size, index):
    """Address of a contiguous vector of `size` elements on the GPU `index`."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == 1 and t.shape[0] == size \
            and t.is_contiguous():
        return t.data_ptr()
    _gpu(t, name, dtype, 1)
    if t.shape[0] != size:
        raise ValueError(f"{name} must have {size} entries (got {t.shape[0]})")
    raise ValueError(f"{name} must be on cuda:{index} (got {t.device})")


def _table(t, index):
    """Address, row stride, rows and columns of a page table."""
    if not isinstance(t, _Tensor) or t.dtype is not _int32_type or t.dim() != 2:
        raise ValueError("page_table must be an int32 tensor of 2 dimension(s)")
    if t.get_device() != index:
        raise ValueError(f"page_table must be on cuda:{index} (got {t.device})")
    batch, max_pages = t.shape
    row, column = t.stride()
    if batch <= 1 or max_pages == 0:
        row = max_pages
    if column != 1 and max_pages > 1 and batch > 0:
        raise ValueError("page_table must be contiguous in its last dimension")
    if row < max_pages:
        raise ValueError("page_table rows must not overlap")
    return t.data_ptr(), row, batch, max_pages


def _pool(page_table, lengths, free, count, page_size):
    """The pool descriptor, checked, with the GPU, the batch and the addresses of lengths and count."""
    _gpu(free, "free", _int32_type, 1)
    index = free.get_device()
    at, stride, batch, max_pages = _table(page_table, index)
    n, c = _vector(lengths, "lengths", _int32_type, batch, index), _vector(count, "count", _int32_type, 2, index)
    return _PoolStruct(at, stride, max_pages, batch, page_size, free.data_ptr(), free.shape[0]), index, batch, n, c


def _on(index, fn, what, *args):
    """Calls a C entry point with the GPU `index` current, on its current stream; a
    status other than OK is raised."""
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
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
    pool, index, batch, n, c = _pool(page_table, lengths, free, count, page_size)
    if not isinstance(done, _Tensor) or done.dtype not in (torch.bool, torch.uint8):
        raise ValueError("done must be a bool or uint8 tensor")
    ended = _vector(done, "done", done.dtype, batch, index)
    common = None if shared is None else _vector(shared, "shared", _int32_type, 1, index)
    if out is None:
        out = (lengths.new_empty(batch), count.new_empty(2))
        to = (out[0].data_ptr(), out[1].data_ptr())
    else:
        to = (_vector(out[0], "out[0]", _int32_type, batch, index), _vector(out[1], "out[1]", _int32_type, 2, index))
    _on(index, lib.int4_cache_release, "int4_cache_release", ctypes.addressof(pool), n, ended, c, common, *to)
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
    ``lengths`` and ``count``.

    A token that lacks a page has none later either. To take such a step back, keep
    ``lengths`` and ``count`` (no ``out``), give pages back with int4_cache_release on
    them, and call again with what that returns."""
    pool, index, batch, n, c = _pool(page_table, lengths, free, count, page_size)
    added = None if new is None else _vector(new, "new", _int32_type, batch, index)
    if rows is None:
        if slots and new is not None and out is None:
            raise ValueError("rows must be given with new")
        rows = batch if new is None else out[2].shape[0] if out is not None and out[2] is not None else 0
    if out is None:
        out = (lengths.new_empty(batch), lengths.new_empty(batch + 1),
               lengths.new_empty(rows, dtype=torch.int64) if slots else None, count.new_empty(2))
        to = [None if t is None else t.data_ptr() for t in out]
    else:
        to = [None if t is None and i == 2 else _vector(t, f"out[{i}]", d, s, index)
              for i, (t, d, s) in enumerate(zip(out, (_int32_type, _int32_type, torch.int64, _int32_type),
                                                (batch, batch + 1, rows, 2)))]
    _on(index, lib.int4_cache_extend, "int4_cache_extend", ctypes.addressof(pool), n, added, c, to[0], to[1], to[2], rows,
        to[3])
    return out


def _rows_of(cache, index, t, name, heads):
    """Rows, row and head stride of a [rows, heads, head_dim] tensor with channels side by side."""
    if isinstance(t, _Tensor) and t.get_device() == index and t.dim() == 3:
        rows, h, d = t.shape
        row, head, channel = t.stride()
        if h == heads and d == cache.head_dim and (channel == 1 or d == 1):
            return rows, row, head
    raise ValueError(_rows_array(cache, t, name, heads))         # (which says what is wrong)


def _rope(rope, index):
    """Address, row stride, positions and rotated channels of a table of cosines and sines, or of none."""
    if rope is None:
        return None, 0, 0, 0
    if not isinstance(rope, _Tensor) or rope.dtype is not torch.float32 or rope.dim() != 2:
        raise ValueError("rope must be a float32 tensor of 2 dimensions")
    if rope.get_device() != index:
        raise ValueError(f"rope must be on cuda:{index} (got {rope.device})")
    positions, rotary = rope.shape
    if positions < 1 or rotary < 2:            # a tensor without elements has no address, which would mean no rotation
        raise ValueError(f"rope must have a position and a pair of channels at least (got {tuple(rope.shape)})")
    row, channel = rope.stride()
    if channel != 1:
        raise ValueError("rope must be contiguous in its last dimension")
    return rope.data_ptr(), row if positions > 1 else rotary, positions, rotary


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
    index = cache.device.index
    q_heads = q.shape[1] if isinstance(q, _Tensor) and q.dim() == 3 else -1
    rows, *qs = _rows_of(cache, index, q, "q", q_heads)
    k_rows, *ks = _rows_of(cache, index, k, "k", cache.heads)
    v_rows, *vs = _rows_of(cache, index, v, "v", cache.heads)
    dtype = q.dtype
    if dtype not in ROWS_DTYPES or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError(f"q, k and v must be float32, float16 or bfloat16, all the same (got {dtype}, {k.dtype}, {v.dtype})")
    if k_rows != rows or v_rows != rows:
        raise ValueError(f"q has {rows} rows, k {k_rows}, v {v_rows}")
    at, stride, batch, max_pages = _table(page_table, index)
    n = _vector(lengths, "lengths", _int32_type, batch, index)
    s = None if starts is None else _vector(starts, "starts", _int32_type, batch + 1, index)
    if s is None and rows != batch:
        raise ValueError(f"without starts there is one row a sequence (got {rows} rows, {batch} sequences)")
    plan = _RowsStruct(at, stride, max_pages, n, s, batch, rows)
    qw = None if q_norm is None else _vector(q_norm, "q_norm", torch.float32, cache.head_dim, index)
    kw = None if k_norm is None else _vector(k_norm, "k_norm", torch.float32, cache.head_dim, index)
    transform = _TransformStruct(qw, kw, eps, *_rope(rope, index), bool(interleaved))
    if out is None:
        out = q.new_empty(q.shape)
    else:
        _gpu(out, "out", dtype, 3)
        if out.shape != q.shape or out.get_device() != index:
            raise ValueError(f"out must be {tuple(q.shape)} on {q.device}")
    _on(index, lib.int4_cache_append, "int4_cache_append", cache._ref, ctypes.addressof(plan), ctypes.addressof(transform),
        q.data_ptr(), *qs, q_heads, k.data_ptr(), *ks, v.data_ptr(), *vs, ROWS_DTYPES[dtype], out.data_ptr())
    return out

"""A paged key/value cache held in 4-bit group codes, and attention over it.

Thin binding over the C ABI in ``include/int4dq_cache.h`` (part of
``libint4dq.so``), in the manner of the package's other calls: torch tensors on
the GPU, work enqueued on ``torch.cuda.current_stream()``, shapes and dtypes
checked here, every step of the computation in the library's HIP kernels.

    cache = Int4Cache.empty(pages, page_size, heads, head_dim, group=128)
    int4_cache_write(cache, k, v, page_table, lengths, starts)
    out = int4_cache_attention(q, cache, page_table, lengths, starts)
    k, v = int4_cache_read(cache, page_table, lengths, starts, rows=...)

The codes of one token and one head are those quantize_int4 (or
quantize_int4_affine) gives for its ``head_dim`` channels as one weight row.

``page_table`` int32 [batch, max_pages], ``lengths`` int32 [batch] (tokens in
the cache, the call's own rows among them) and ``starts`` int32 [batch + 1]
say which rows are whose: sequence b owns rows starts[b] .. starts[b+1]-1, its
last tokens. Without ``starts`` there is one row a sequence, the form of token
generation. All three live on the GPU and are read there, so a captured graph
replays with what they hold at that time. Rows that no sequence owns (a padded
batch) stay as they were in an ``out`` tensor that the caller passes; in one
made by the call they hold nothing of meaning.
"""
from __future__ import annotations

import ctypes

import torch

from . import _gpu, _raise, lib

__all__ = ["Int4Cache", "int4_cache_write", "int4_cache_read", "int4_cache_attention",
           "cache_attention_workspace_bytes", "cache_attention_workspace"]

ROWS_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

_i64, _vp, _int, _f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float


class _CacheStruct(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k_packed", "k_scales", "k_zeros", "v_packed", "v_scales", "v_zeros")] + \
               [(n, _i64) for n in ("pages", "page_size", "heads", "head_dim", "group")]


class _RowsStruct(ctypes.Structure):
    _fields_ = [("page_table", _vp), ("table_stride", _i64), ("max_pages", _i64), ("lengths", _vp), ("starts", _vp),
                ("batch", _i64), ("rows", _i64)]


# Every function declared in include/int4dq_cache.h, with its ctypes signature.
CACHE_SIGNATURES = {
    "int4_cache_row_bytes": (_i64, [_i64]),
    "int4_cache_write": (_int, [_vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _int, _vp]),
    "int4_cache_read": (_int, [_vp, _vp, _vp, _vp, _int, _vp]),
    "int4_cache_attention": (_int, [_vp, _vp, _vp, _i64, _i64, _int, _i64, _f32, _int, _i64, _vp, _vp, _vp, _i64,
                                    _vp]),
    "int4_cache_attention_workspace_bytes": (_i64, [_vp, _vp, _i64]),
}
for _name, (_res, _args) in CACHE_SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


try:                                    # a quarter of the time of current_stream(device).cuda_stream
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


class Int4Cache:
    """The tensors of a cache (layouts: include/int4dq_cache.h) as one handle.

    k_packed uint8 [pages, heads, page_size, row_bytes], v_packed uint8 [pages,
    heads, page_size / 16, row_bytes, 16], k_scales and v_scales float16 [pages,
    heads, page_size / 16, groups, 16], and for affine codes k_zeros and v_zeros
    uint8 of the scales' shape. The handle keeps the tensors alive and writes to
    them in place; they must not be resized while it is in use."""

    __slots__ = ("k_packed", "k_scales", "v_packed", "v_scales", "k_zeros", "v_zeros", "pages", "page_size", "heads",
                 "head_dim", "group", "device", "_struct", "_ref")

    def __init__(self, k_packed: torch.Tensor, k_scales: torch.Tensor, v_packed: torch.Tensor,
                 v_scales: torch.Tensor, head_dim: int, group: int = 128, k_zeros: torch.Tensor | None = None,
                 v_zeros: torch.Tensor | None = None):
        row = lib.int4_cache_row_bytes(head_dim)
        if row < 0:
            raise ValueError(f"head_dim must be 1 to 256 (got {head_dim})")
        if group < 1 or (group < head_dim and group not in (32, 64, 128)):
            raise ValueError(f"group must be 32, 64 or 128, or at least head_dim (got {group})")
        if (k_zeros is None) != (v_zeros is None):
            raise ValueError("k_zeros and v_zeros must both be given or both be None")
        _gpu(k_packed, "k_packed", torch.uint8, 4)
        pages, heads, page_size, _ = k_packed.shape
        if page_size < 16 or page_size & (page_size - 1):
            raise ValueError(f"page_size must be a power of two from 16 up (got {page_size})")
        units = (pages, heads, page_size // 16)
        G = -(-head_dim // group)
        for name, t, dtype, shape in (("k_packed", k_packed, torch.uint8, (pages, heads, page_size, row)),
                                      ("v_packed", v_packed, torch.uint8, (*units, row, 16)),
                                      ("k_scales", k_scales, torch.float16, (*units, G, 16)),
                                      ("v_scales", v_scales, torch.float16, (*units, G, 16)),
                                      ("k_zeros", k_zeros, torch.uint8, (*units, G, 16)),
                                      ("v_zeros", v_zeros, torch.uint8, (*units, G, 16))):
            if t is None and name.endswith("zeros"):
                continue
            _gpu(t, name, dtype, len(shape))
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
            if t.device != k_packed.device:
                raise ValueError(f"{name} must be on {k_packed.device}")
        self.k_packed, self.k_scales, self.k_zeros = k_packed, k_scales, k_zeros
        self.v_packed, self.v_scales, self.v_zeros = v_packed, v_scales, v_zeros
        self.pages, self.page_size, self.heads, self.head_dim, self.group = pages, page_size, heads, head_dim, group
        self.device = k_packed.device
        ptr = [None if t is None else t.data_ptr() for t in (k_packed, k_scales, k_zeros, v_packed, v_scales, v_zeros)]
        self._struct = _CacheStruct(*ptr, pages, page_size, heads, head_dim, group)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, group: int = 128, affine: bool = False,
              device="cuda") -> "Int4Cache":
        """A cache with room for ``pages`` pages, its contents undefined until written."""
        row = lib.int4_cache_row_bytes(head_dim)
        if row < 0 or group < 1 or pages < 1 or heads < 1:
            raise ValueError(f"invalid sizes pages={pages} heads={heads} head_dim={head_dim} group={group}")
        if page_size < 16 or page_size & (page_size - 1):
            raise ValueError(f"page_size must be a power of two from 16 up (got {page_size})")
        units = (pages, heads, page_size // 16)
        G = -(-head_dim // group)

        def new(*shape, dtype=torch.uint8):
            return torch.empty(shape, dtype=dtype, device=device)

        return cls(new(pages, heads, page_size, row), new(*units, G, 16, dtype=torch.float16), new(*units, row, 16),
                   new(*units, G, 16, dtype=torch.float16), head_dim, group,
                   new(*units, G, 16) if affine else None, new(*units, G, 16) if affine else None)

    @property
    def affine(self) -> bool:
        return self.k_zeros is not None

    def nbytes(self) -> int:
        """Bytes of device memory the cache takes."""
        return sum(t.numel() * t.element_size() for t in (self.k_packed, self.k_scales, self.k_zeros, self.v_packed,
                                                          self.v_scales, self.v_zeros) if t is not None)


def _is_cache(cache):
    if not isinstance(cache, Int4Cache):
        raise ValueError("cache must be an Int4Cache")


def _int32(cache, name, t, ndim):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != ndim:
        raise ValueError(f"{name} must be an int32 tensor of {ndim} dimension(s)")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device} (got {t.device})")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _plan(cache, page_table, lengths, starts, rows):
    """The rows descriptor, checked; rows: what the row-wise arrays hold."""
    _int32(cache, "page_table", page_table, 2)
    _int32(cache, "lengths", lengths, 1)
    batch, max_pages = page_table.shape
    if lengths.shape[0] != batch:
        raise ValueError(f"lengths has {lengths.shape[0]} entries, page_table {batch} rows")
    sp = None
    if starts is not None:
        _int32(cache, "starts", starts, 1)
        if starts.shape[0] != batch + 1:
            raise ValueError(f"starts has {starts.shape[0]} entries, a batch of {batch} needs {batch + 1}")
        sp = starts.data_ptr()
    elif rows != batch:
        raise ValueError(f"without starts there is one row a sequence (got {rows} rows, {batch} sequences)")
    stride = page_table.stride(0) if batch > 1 else max_pages
    if stride < max_pages:
        raise ValueError("page_table rows must not overlap")
    return _RowsStruct(page_table.data_ptr(), stride, max_pages, lengths.data_ptr(), sp, batch, rows)


def _rows_array(cache, t, name, heads):
    """Checks a [rows, heads, head_dim] tensor with channels side by side; its row
    and head strides."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != cache.head_dim:
        raise ValueError(f"{name} must be a tensor [rows, {heads}, {cache.head_dim}]"
                         + (f" (got {tuple(t.shape)})" if isinstance(t, torch.Tensor) else ""))
    if t.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device} (got {t.device})")
    row, head, channel = t.stride()
    if channel != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return row, head


def _call(cache, fn, what, *args):
    """Calls a C entry point with the cache's device current, on that device's
    current stream; a status other than OK is raised."""
    index = cache.device.index
    if torch.cuda.current_device() == index:
        rc = fn(cache._ref, *args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(cache._ref, *args, _raw_stream(index))
    if rc:
        _raise(rc, what)


def int4_cache_write(cache: Int4Cache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                     lengths: torch.Tensor, starts: torch.Tensor | None = None) -> None:
    """Quantise k and v [rows, heads, head_dim] (float32, float16 or bfloat16, any
    row and head strides) into the cache at the rows' positions."""
    _is_cache(cache)
    ks, vs = _rows_array(cache, k, "k", cache.heads), _rows_array(cache, v, "v", cache.heads)
    if k.dtype not in ROWS_DTYPES or v.dtype != k.dtype:
        raise ValueError(f"k and v must be float32, float16 or bfloat16, both the same (got {k.dtype}, {v.dtype})")
    if v.shape[0] != k.shape[0]:
        raise ValueError(f"k has {k.shape[0]} rows, v {v.shape[0]}")
    plan = _plan(cache, page_table, lengths, starts, k.shape[0])
    _call(cache, lib.int4_cache_write, "int4_cache_write", ctypes.addressof(plan), k.data_ptr(), *ks, v.data_ptr(), *vs,
          ROWS_DTYPES[k.dtype])


def int4_cache_read(cache: Int4Cache, page_table: torch.Tensor, lengths: torch.Tensor,
                    starts: torch.Tensor | None = None, *, rows: int | None = None,
                    dtype: torch.dtype = torch.float16, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """Keys and values [rows, heads, head_dim] of ``dtype`` at the rows' positions:
    the last starts[b+1] - starts[b] tokens of each sequence (all of them where
    that is lengths[b]). ``rows`` is starts[batch], known to the caller (default:
    one row a sequence); ``out``: a pair of contiguous tensors to fill."""
    _is_cache(cache)
    if dtype not in ROWS_DTYPES:
        raise ValueError(f"dtype must be float32, float16 or bfloat16 (got {dtype})")
    if rows is None:
        if starts is not None and out is None:
            raise ValueError("rows must be given with starts")
        rows = out[0].shape[0] if out is not None else page_table.shape[0]
    plan = _plan(cache, page_table, lengths, starts, rows)
    shape = (rows, cache.heads, cache.head_dim)
    if out is None:
        out = torch.empty((2, *shape), dtype=dtype, device=cache.device).unbind(0)
    else:
        for name, t in zip(("out[0]", "out[1]"), out):
            _gpu(t, name, dtype, 3)
            if tuple(t.shape) != shape or t.device != cache.device:
                raise ValueError(f"{name} must be {shape} on {cache.device}")
    _call(cache, lib.int4_cache_read, "int4_cache_read", ctypes.addressof(plan), out[0].data_ptr(), out[1].data_ptr(),
          ROWS_DTYPES[dtype])
    return out


def _workspace_bytes(cache, plan, q_heads):
    n = lib.int4_cache_attention_workspace_bytes(cache._ref, ctypes.addressof(plan), q_heads)
    if n < 0:
        raise ValueError(lib.int4_last_error().decode())
    return n


def cache_attention_workspace_bytes(cache: Int4Cache, batch: int, rows: int, q_heads: int) -> int:
    """Bytes of workspace int4_cache_attention uses for these sizes: ``rows`` rows
    of ``q_heads`` query heads over ``batch`` sequences, whatever their page tables
    (a call whose table is short takes less, or none)."""
    _is_cache(cache)
    one = None if rows == batch else 1
    most = 2 ** 31 - 1
    return _workspace_bytes(cache, _RowsStruct(None, most, most, None, one, batch, rows), q_heads)


def cache_attention_workspace(cache: Int4Cache, batch: int, rows: int, q_heads: int) -> torch.Tensor:
    """A workspace tensor for int4_cache_attention(..., workspace=)."""
    return torch.empty(cache_attention_workspace_bytes(cache, batch, rows, q_heads), dtype=torch.uint8,
                       device=cache.device)


def int4_cache_attention(q: torch.Tensor, cache: Int4Cache, page_table: torch.Tensor, lengths: torch.Tensor,
                         starts: torch.Tensor | None = None, *, scale: float | None = None, causal: bool = True,
                         window: int = 0, return_lse: bool = False, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None):
    """Softmax attention of q [rows, q_heads, head_dim] (float16 or bfloat16, any
    row and head strides) over the cache: out of q's shape and dtype, and with
    ``return_lse`` the logarithm of each softmax sum, float32 [rows, q_heads].

    Query head h reads key/value head h // (q_heads / heads). A row sees the keys
    of its sequence up to its own position (``causal``; its own key is written
    before), the last ``window`` of them where that is not 0, or all of them. A
    row that sees none gets 0 and an lse of -infinity. ``scale`` multiplies the
    scores (default head_dim ** -0.5). ``workspace``: a uint8 tensor from
    cache_attention_workspace; without one the call takes its scratch from
    torch's allocator."""
    _is_cache(cache)
    q_heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
    qs = _rows_array(cache, q, "q", q_heads)
    if q.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"q must be float16 or bfloat16 (got {q.dtype})")
    if q_heads < 1 or q_heads % cache.heads:
        raise ValueError(f"q has {q_heads} heads, which is no multiple of the cache's {cache.heads}")
    rows = q.shape[0]
    plan = _plan(cache, page_table, lengths, starts, rows)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _gpu(out, "out", q.dtype, 3)
        if tuple(out.shape) != tuple(q.shape) or out.device != q.device:
            raise ValueError(f"out must be {tuple(q.shape)} on {q.device}")
    lse = torch.empty((rows, q_heads), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        n = _workspace_bytes(cache, plan, q_heads)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    else:
        _gpu(workspace, "workspace", torch.uint8, 1)
        if workspace.device != q.device:
            raise ValueError(f"workspace must be on {q.device}")
        n = workspace.numel()
    _call(cache, lib.int4_cache_attention, "int4_cache_attention", ctypes.addressof(plan), q.data_ptr(), *qs,
          ROWS_DTYPES[q.dtype], q_heads, cache.head_dim ** -0.5 if scale is None else scale, bool(causal), int(window),
          out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr() if n else None, n)
    return (out, lse) if return_lse else out

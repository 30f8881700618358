"""The C ABI and Python binding of a serving step over the 4-bit cache where no GPU
is needed: what the calls refuse, before anything is enqueued."""
import ctypes
import re
from pathlib import Path

import pytest
import torch

import dequantizing_gemm_amd as dq
from dequantizing_gemm_amd import cache, cache_step

ROOT = Path(__file__).resolve().parents[1]
P = 4096                                       # an address that is never read: every call here is refused


def test_header_and_binding_name_the_same_functions():
    text = re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "int4dq_cache_step.h").read_text(), flags=re.S)
    declared = set(re.findall(r"\b(int4_cache_\w+)\s*\(", text))
    assert declared == set(cache_step.CACHE_STEP_SIGNATURES)
    assert all(hasattr(dq.lib, name) for name in declared)
    for name in cache_step.__all__:
        assert getattr(dq, name) is getattr(cache_step, name) and name in dq.__all__


def refused(rc, needle, what):
    assert rc == dq.EINVAL
    text = dq.lib.int4_last_error().decode()
    assert needle in text and what in text, text


POOL = dict(page_table=P, table_stride=8, max_pages=8, batch=3, page_size=64, free=P, pages=50)
BAD_POOL = [(dict(page_size=8), "page_size"), (dict(page_size=48), "page_size"), (dict(page_size=1 << 21), "page_size"),
            (dict(pages=-1), "pages"), (dict(pages=1 << 31), "pages"), (dict(batch=-1), "batch"),
            (dict(batch=(1 << 22) + 1), "batch"), (dict(table_stride=7), "table_stride"), (dict(max_pages=-1), "max_pages"),
            (dict(max_pages=1 << 31, table_stride=1 << 31), "max_pages"), (dict(table_stride=1 << 41), "table_stride"),
            (dict(page_table=None), "non-NULL"), (dict(free=None), "non-NULL")]


@pytest.mark.parametrize("change,needle", BAD_POOL)
def test_pools_refused(change, needle):
    pool = cache_step._PoolStruct(**{**POOL, **change})
    at = ctypes.addressof(pool)
    refused(dq.lib.int4_cache_release(at, P, P, P, None, P, P, None), needle, "int4_cache_release")
    refused(dq.lib.int4_cache_extend(at, P, None, P, P, P, P, 5, P, None), needle, "int4_cache_extend")


def test_page_calls_refused():
    pool = cache_step._PoolStruct(**POOL)
    at, L = ctypes.addressof(pool), dq.lib
    for a in ((None, P, P, P, None, P, P), (at, None, P, P, None, P, P), (at, P, None, P, None, P, P),
              (at, P, P, None, None, P, P), (at, P, P, P, None, None, P), (at, P, P, P, None, P, None)):
        refused(L.int4_cache_release(*a, None), "non-NULL", "int4_cache_release")
    for a in ((None, P, P, P, P, P, P, 5, P), (at, None, P, P, P, P, P, 5, P), (at, P, P, None, P, P, P, 5, P),
              (at, P, P, P, None, P, P, 5, P), (at, P, P, P, P, None, P, 5, P), (at, P, P, P, P, P, P, 5, None)):
        refused(L.int4_cache_extend(*a, None), "non-NULL", "int4_cache_extend")
    for rows in (-1, (1 << 26) + 1):
        refused(L.int4_cache_extend(at, P, P, P, P, P, P, rows, P, None), "rows", "int4_cache_extend")


CACHE = dict(k_packed=P, k_scales=P, k_zeros=None, v_packed=P, v_scales=P, v_zeros=None, pages=9, page_size=16, heads=2,
             head_dim=128, group=64)
ROWS = dict(page_table=P, table_stride=4, max_pages=4, lengths=P, starts=P, batch=3, rows=7)
TURN = dict(q_norm=P, k_norm=P, eps=1e-6, rope=P, rope_stride=128, rope_positions=100, rotary_dim=128, interleaved=0)


def append(c={}, r={}, t={}, q=P, q_heads=4, k=P, v=P, dtype=2, out=P, strides=(512, 128, 256, 128, 256, 128), turn=True):
    cs, rs = cache._CacheStruct(**{**CACHE, **c}), cache._RowsStruct(**{**ROWS, **r})
    ts = cache_step._TransformStruct(**{**TURN, **t})
    s = strides
    return dq.lib.int4_cache_append(ctypes.addressof(cs), ctypes.addressof(rs), ctypes.addressof(ts) if turn else None, q,
                                    s[0], s[1], q_heads, k, s[2], s[3], v, s[4], s[5], dtype, out, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(c=dict(head_dim=0)), "head_dim"), (dict(c=dict(group=48)), "group"), (dict(c=dict(k_scales=None)), "non-NULL"),
    (dict(c=dict(v_zeros=P)), "both"), (dict(c=dict(k_packed=P + 8)), "aligned"), (dict(r=dict(rows=-1)), "rows"),
    (dict(r=dict(starts=None)), "one row a sequence"), (dict(r=dict(lengths=None)), "lengths"),
    (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(q_heads=0), "q_heads"), (dict(q_heads=65536), "q_heads"),
    (dict(r=dict(rows=1 << 24)), "2^25"), (dict(r=dict(batch=1 << 20)), "2^20"),
    (dict(turn=False), "transform"), (dict(t=dict(eps=-1.0)), "eps"), (dict(t=dict(eps=float("nan"))), "eps"),
    (dict(t=dict(eps=float("inf"))), "eps"), (dict(t=dict(rotary_dim=0)), "rotary_dim"),
    (dict(t=dict(rotary_dim=63)), "rotary_dim"), (dict(t=dict(rotary_dim=130)), "rotary_dim"),
    (dict(t=dict(rope_positions=0)), "rope_positions"), (dict(t=dict(rope_stride=127)), "rope_stride"),
    (dict(t=dict(rope_stride=(1 << 30) + 1)), "rope_stride"), (dict(q=None), "non-NULL"), (dict(k=None), "non-NULL"),
    (dict(v=None), "non-NULL"), (dict(out=None), "non-NULL"), (dict(strides=(1 << 31, 1, 1, 1, 1, 1)), "stride"),
    (dict(strides=(1, 1, 1, 1, 1, -1 << 31)), "stride")])
def test_append_refused(kw, needle):
    refused(append(**kw), needle, "int4_cache_append")


def test_append_of_nothing():
    """No rows or no sequences: nothing to do, no pointer needed."""
    assert append(r=dict(rows=0), q=None, k=None, v=None, out=None) == dq.OK
    assert append(r=dict(rows=0, batch=0, lengths=None), q=None, k=None, v=None, out=None) == dq.OK


def test_tensors_refused():
    """Shapes, types and devices, before any pointer is passed on."""
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    free, count = torch.zeros(9, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: dq.int4_cache_release(t, n, free, count, 16, n.bool()),
                 lambda: dq.int4_cache_extend(t, n, free, count, 16),
                 lambda: dq.int4_cache_extend(t, n, None, count, 16)):
        with pytest.raises(ValueError, match="free"):
            call()
    q = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="cache"):
        dq.int4_cache_append(None, q, q, q, t, n)

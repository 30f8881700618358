"""The 4-bit cache's C ABI and Python binding where no GPU is needed."""
import re
from pathlib import Path

import pytest
import torch

import dequantizing_gemm_amd as dq
from dequantizing_gemm_amd import cache

ROOT = Path(__file__).resolve().parents[1]


def test_header_and_binding_name_the_same_functions():
    text = re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "int4dq_cache.h").read_text(), flags=re.S)
    declared = set(re.findall(r"\b(int4_cache_\w+)\s*\(", text))
    assert declared == set(cache.CACHE_SIGNATURES)
    assert all(hasattr(dq.lib, name) for name in declared)
    for name in cache.__all__:
        assert getattr(dq, name) is getattr(cache, name)


@pytest.mark.parametrize("head_dim,width", [(1, 32), (64, 32), (65, 48), (96, 48), (97, 64), (128, 64), (129, 96),
                                            (192, 96), (193, 128), (256, 128), (0, -1), (-5, -1), (257, -1)])
def test_row_bytes(head_dim, width):
    assert dq.lib.int4_cache_row_bytes(head_dim) == width


def test_workspace_bytes():
    """Sizes only: grows with the query heads' tiles, 0 where no table can hold more
    than a block's least share, -1 with a message for what attention refuses."""
    import ctypes
    c = cache._CacheStruct(None, None, None, None, None, None, 100, 64, 8, 128, 128)

    def size(batch, rows, q_heads, max_pages=1000, starts=1):
        r = cache._RowsStruct(None, max_pages, max_pages, None, starts, batch, rows)
        return dq.lib.int4_cache_attention_workspace_bytes(ctypes.addressof(c), ctypes.addressof(r), q_heads)

    assert 0 < size(4, 4, 32) < size(1, 500, 32) < 1 << 30
    assert size(4, 4, 32, max_pages=16) == 0 < size(4, 4, 32, max_pages=17)
    assert size(0, 0, 32) == 0 and size(4, 0, 32) == 0
    assert size(65, 65, 32) > size(64, 64, 32)              # the plan of a large batch
    for bad in ((4, 4, 12), (4, 4, 0), (-1, 4, 32), (4, 1 << 30, 32)):
        assert size(*bad) == -1 and dq.lib.int4_last_error()
    assert size(3, 4, 32, starts=None) == -1


def test_tensors_elsewhere_are_refused():
    k = torch.zeros(1, 1, 16, 32, dtype=torch.uint8)
    v = torch.zeros(1, 1, 1, 32, 16, dtype=torch.uint8)
    s = torch.zeros(1, 1, 1, 1, 16, dtype=torch.float16)
    with pytest.raises(ValueError, match="k_packed"):
        dq.Int4Cache(k, s, v, s, 64)
    with pytest.raises(ValueError, match="head_dim"):
        dq.Int4Cache(k, s, v, s, 300)
    with pytest.raises(ValueError, match="group"):
        dq.Int4Cache(k, s, v, s, 128, 48)
    t = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        dq.int4_cache_write(None, k, k, t, t[0])
    with pytest.raises(ValueError):
        dq.int4_cache_attention(k, None, t, t[0])

"""What the calls of a serving step over the 4-bit cache refuse with tensors on the GPU, and that
nothing is written then."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def dq():
    import dequantizing_gemm_amd as dq
    return dq


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("shape", [(0, 64), (9, 0), (9, 1)])
def test_ropes_without_elements(dq, shape):
    cache = dq.Int4Cache.empty(1, 16, 1, 64, 64)
    cache.k_packed.fill_(0x77)
    q = torch.ones(1, 1, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    with pytest.raises(ValueError, match="rope"):
        dq.int4_cache_append(cache, q, q, q, i32(0)[None], i32(3), rope=torch.ones(9, 64, device=DEV)[:shape[0], :shape[1]], out=out)
    assert (out == 7).all() and (cache.k_packed == 0x77).all()

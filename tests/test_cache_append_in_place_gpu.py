"""int4_cache_append on MI355X with queries in place, in calls of every size: the same bits as into
another tensor, keys and values that lie behind the queries in memory untouched."""
import pytest
import torch

from tests.test_cache_gpu import BF16, DEV, F16, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 37, 4100])
@pytest.mark.parametrize("D,rotary,interleaved,dtype,off", [(128, 128, False, BF16, 0), (128, 128, False, BF16, 1), (64, 32, False, F16, 0),
                                                            (96, 96, True, F32, 0), (250, 250, False, F16, 0), (33, 20, False, F32, 0)])
def test_queries_in_place(D, rotary, interleaved, dtype, off, rows):
    import dequantizing_gemm_amd as dq
    H, HQ, S = 8, 32, 64
    g = torch.Generator(device=DEV).manual_seed(D + rows)
    n = rows * HQ * D
    memory = torch.randn(off + n + 2 * rows * H * D, generator=g, device=DEV).to(dtype)
    whole = memory.clone()
    q = memory[off:off + n].view(rows, HQ, D)
    k, v = memory[off + n:].view(2, rows, H, D)
    angle = torch.rand(rows + 9, rotary // 2, generator=g, device=DEV)
    kw = dict(q_norm=torch.rand(D, generator=g, device=DEV) + 0.5, k_norm=torch.rand(D, generator=g, device=DEV) + 0.5,
              rope=torch.cat([angle.cos(), angle.sin()], 1), interleaved=interleaved)
    pages = -(-rows // S)
    plan = (torch.arange(pages, dtype=torch.int32, device=DEV)[None], torch.tensor([rows], dtype=torch.int32, device=DEV),
            torch.tensor([0, rows], dtype=torch.int32, device=DEV))
    caches = [dq.Int4Cache.empty(pages, S, H, D, 32) for _ in range(2)]
    names = ("k_packed", "v_packed", "k_scales", "v_scales")
    for c in caches:
        for x in names:
            getattr(c, x).zero_()
    print("case: in place", D, rotary, interleaved, dtype, off, rows, flush=True)
    want = dq.int4_cache_append(caches[0], q, k, v, *plan, **kw)
    assert torch.equal(memory, whole)
    got = dq.int4_cache_append(caches[1], q, k, v, *plan, out=q, **kw)
    assert got is q and torch.equal(got, want)
    assert torch.equal(memory[:off], whole[:off]) and torch.equal(memory[off + n:], whole[off + n:])
    for x in names:
        assert torch.equal(getattr(caches[0], x), getattr(caches[1], x)), x

"""The Python binding of a serving step over the 4-bit cache where no GPU is needed: arguments
whose addresses would mean something else are refused before any is taken."""
import pytest
import torch

from dequantizing_gemm_amd import cache_step

CPU = -1                                       # what Tensor.get_device says of these tensors


@pytest.mark.parametrize("shape", [(0, 64), (9, 0), (0, 0), (9, 1)])
def test_a_rope_without_elements_is_not_no_rope(shape):
    """Its address is NULL, which says that nothing is rotated."""
    rope = torch.zeros(shape)
    assert rope.numel() > 0 or rope.data_ptr() == 0
    with pytest.raises(ValueError, match="rope"):
        cache_step._rope(rope, CPU)
    with pytest.raises(ValueError, match="rope"):
        cache_step._rope(torch.zeros(9, 64)[:shape[0], :shape[1]], CPU)


def test_ropes():
    assert cache_step._rope(None, CPU) == (None, 0, 0, 0)
    rope = torch.zeros(9, 80)
    assert cache_step._rope(rope[:, :64], CPU) == (rope.data_ptr(), 80, 9, 64)
    assert cache_step._rope(rope[3:4], CPU) == (rope[3].data_ptr(), 80, 1, 80)
    for bad in (rope.double(), rope[0], rope.t(), 5, rope[:, ::2]):
        with pytest.raises(ValueError, match="rope"):
            cache_step._rope(bad, CPU)
    with pytest.raises(ValueError, match="rope"):
        cache_step._rope(rope, 0)

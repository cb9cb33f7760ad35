"""Rotary positions at the ends of what fa_rope takes."""
import pytest
import torch

import exact_io_aware_52_b200 as fa
from exact_io_aware_52_b200 import _binding as fb

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("d,dim", [(64, 64), (50, 20)])  # slots of 16 components; element by element
def test_positions_at_the_ends_of_int32(d, dim):
    """pos0 gives what the same positions in a tensor give, up to the last one; past it the call is refused."""
    q = torch.randn(1, 2, 8, d, generator=torch.Generator().manual_seed(70)).to(BF16).to(dev())
    r = fa.Rotary(dim)
    for pos0 in (2 ** 31 - 8, -(2 ** 31), -3):
        pos = (torch.arange(8, dtype=torch.int64) + pos0).to(torch.int32).to(dev())
        assert torch.equal(fa.rope(r, q, pos0=pos0), fa.rope(r, q, pos=pos))
    for pos0 in (2 ** 31 - 7, 2 ** 31 - 1):
        with pytest.raises(fb.FaError):
            fa.rope(r, q, pos0=pos0)
    assert fa.rope(r, q[:, :, :1], pos0=2 ** 31 - 1).shape == (1, 2, 1, d)

"""Attention over the 8-bit cache at the ends of what its scales may be."""
import pytest
import torch

import exact_io_aware_52_b200 as fa
from tests import serving_check as chk
from tests import serving_ref as ref
from tests.test_serving_gpu import run_attention

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("d,H,page", [(64, 3, 16), (128, 16, 64), (256, 5, 32)])
@pytest.mark.parametrize("lens", [[300, 40], [9000, 300]])  # clusters; split keys, whole pairs and their merge
@pytest.mark.parametrize("exp", [-149, -127, -121, -113, -100, 0, 60])
def test_value_scales_of_any_size(exp, lens, d, H, page, out_dtype):
    """One scale for all values, down to the smallest fp32 number: O is as exact as with a scale of 1."""
    pool = ref.pool(50 + d, lens, 1, page, d)
    pool[3].fill_(2.0 ** exp)
    q = torch.randn(2, H, 1, d, generator=torch.Generator().manual_seed(51)).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.05, out_dtype)
    chk.check(o, lse, q, pool, lens, True, 0.05, page)


@pytest.mark.parametrize("lens", [[300], [9000]])
def test_value_scales_at_the_upper_end(lens):
    """Codes of at most 1 times 2^86: sums over the keys of what is not yet divided stay within fp32."""
    pool = ref.pool(52, lens, 1, 64, 128)
    pool[1].copy_((pool[1].float() / 448).to(ref.E4M3))
    pool[3].fill_(2.0 ** 86)
    q = torch.randn(1, 4, 1, 128, generator=torch.Generator().manual_seed(53)).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.05)
    chk.check(o, lse, q, pool, lens, True, 0.05, 64)

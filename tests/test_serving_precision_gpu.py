"""The precision of attention over the 8-bit cache with few keys, where nothing averages a weight's rounding away."""
import pytest
import torch

from tests import serving_check as chk
from tests import serving_ref as ref
from tests.test_serving_gpu import run_attention

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("room", [1, 400])  # taken whole; split keys
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,N", [(1, 1), (4, 1), (5, 1), (8, 1), (4, 3), (16, 1), (33, 1)])
def test_fp32_outputs_keep_fp32_weights(H, N, d, room):
    """Scores of 0.01 and less, so that their own error is below 2^-22: O is then within about 2^-16 of its terms, 32
    times less than a weight rounded to fp16 may be off."""
    lens = [2, 3, 5, 17, 1, 40]
    pool = ref.pool(100 + d, lens, 1, 16, d)
    q = torch.randn(len(lens), H, N, d, generator=torch.Generator().manual_seed(101)).to(BF16)
    wide = (*pool[:4], torch.cat([pool[4]] + [torch.full_like(pool[4], -1)] * (room - 1), 1))
    scale = 2.0 ** -10
    o, lse = run_attention(q, wide, lens, False, scale)
    t = chk.attend_terms(q, pool, lens, False, scale, 16)
    assert (chk.bounds(t, F32)[0] <= 2.0 ** -15 * (t["oabs"] + t["o"].abs()) + t["codes"] * 2.0 ** -36).all()
    assert chk.off(o, lse, t) is None

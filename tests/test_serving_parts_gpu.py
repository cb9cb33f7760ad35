"""Attention over the 8-bit cache with every part of a split seen in the outputs, and with bounds for each row."""
import pytest
import torch

from tests import serving_check as chk
from tests import serving_ref as ref
from tests.test_serving_gpu import ATTN_SHAPES, run_attention

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("H,N,d,lens", [
    (2, 1, 64, [70_001]), (2, 1, 64, [40_000, 3, 25_000]), (2, 1, 64, [129] * 67), (8, 1, 128, [70_001]),
    (4, 1, 128, [9000, 17, 30_000]), (16, 1, 128, [20_011]), (8, 1, 256, [20_011, 400]), (5, 4, 64, [12_345, 8000]),
    (4, 7, 128, [6000]), (4, 1, 128, [2000]), (12, 1, 64, [1000, 999])])
@pytest.mark.parametrize("block", [16, 64])
def test_every_part_counts(H, N, d, lens, block, out_dtype):
    """A part of `block` tokens left out, weighed wrongly or counted twice shows in its components; that these bounds
    see it is tested on the CPU."""
    pool = chk.stripe_values(ref.pool(81, lens, 1, 128, d), lens, 128, block)
    q = torch.randn(len(lens), H, N, d, generator=torch.Generator().manual_seed(82)).to(BF16)
    o, lse = run_attention(q, pool, lens, True, chk.STRIPE_SCALE, out_dtype)
    chk.check(o, lse, q, pool, lens, True, chk.STRIPE_SCALE, 128)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", ATTN_SHAPES)
def test_rows_within_their_own_bounds(shape, causal):
    H, H_kv, N, d, page, lens = shape
    pool = ref.pool(83, lens, H_kv, page, d)
    q = torch.randn(len(lens), H, N, d, generator=torch.Generator().manual_seed(84)).to(BF16)
    o, lse = run_attention(q, pool, lens, causal, d ** -0.5)
    chk.check(o, lse, q, pool, lens, causal, d ** -0.5, page)


@pytest.mark.parametrize("lens", [[70_001], [40_000, 3, 25_000], [129] * 67])
def test_many_parts_within_their_own_bounds(lens):
    pool = ref.pool(32, lens, 1, 128, 64)
    q = torch.randn(len(lens), 2, 1, 64, generator=torch.Generator().manual_seed(30)).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.125)
    chk.check(o, lse, q, pool, lens, True, 0.125, 128)


def test_scales_far_apart_within_their_own_bounds():
    """Keys whose page has a small value scale next to pages with a large one."""
    lens = [300, 5000]
    pool = ref.pool(34, lens, 2, 16, 64, spread=(-30, 20))
    pool[2].copy_(0.01 + 0.02 * torch.rand(pool[2].shape, generator=torch.Generator().manual_seed(85)))
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(86)).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.125)
    chk.check(o, lse, q, pool, lens, True, 0.125, 16)

"""The bounds that attention over the 8-bit cache is held to reject what they have to: parts left out, weighed
wrongly or counted twice."""
import pytest
import torch

from tests import serving_check as chk
from tests import serving_ref as ref


@pytest.mark.parametrize("n,block", [(70_001, 64), (9000, 64), (9000, 16)])
def test_bounds_reject_a_part_left_out(n, block):
    pool = chk.stripe_values(ref.pool(32, [n], 1, 128, 64), [n], 128, block)
    q = torch.randn(1, 2, 1, 64, generator=torch.Generator().manual_seed(30)).to(torch.bfloat16)
    scale = chk.STRIPE_SCALE
    t = chk.attend_terms(q, pool, [n], True, scale, 128)
    o, lse = t["o"].float(), t["lse"].float()
    assert chk.off(o, lse, t) is None
    assert chk.off(o.bfloat16(), lse, t) is None
    x = torch.einsum("hd,nd->hn", q[0, :, 0].double(), ref.dense(pool[0].float(), pool[2], pool[4], 0, n, 128)[0]) * scale
    p = torch.softmax(x, -1)
    v = ref.dense(pool[1].float(), pool[3], pool[4], 0, n, 128)[0]
    blocks = -(-n // block)
    for i in torch.linspace(0, blocks - 2, 23).long().tolist():  # the last one may be a few tokens
        part = torch.einsum("hn,nd->hd", p[:, i * block:(i + 1) * block], v[i * block:(i + 1) * block])[None, :, None]
        for wrong in (t["o"] - part, t["o"] + part, t["o"] + part / 8):
            assert chk.off(wrong.float(), lse, t) is not None
    # a whole row off by more than a few roundings of its weights
    assert chk.off((t["o"] * (1 + 2.0 ** -8)).float(), lse, t) is not None


def test_bounds_reject_rows_of_zeros():
    n = 70_001
    pool = ref.pool(32, [n], 1, 128, 64)
    q = torch.randn(1, 2, 1, 64, generator=torch.Generator().manual_seed(30)).to(torch.bfloat16)
    t = chk.attend_terms(q, pool, [n], True, 0.125, 128)
    assert chk.off(t["o"].float(), t["lse"].float(), t) is None
    near = (t["o"].abs() <= chk.bounds(t, torch.float32)[0]).double().mean()
    assert near < 0.01  # components that could be 0 instead

"""Appending turned keys at full width: the sines of a whole page in more than 48 KB of shared memory, pages that
are read twice, and the scales that follow.

A turned component errs by delta = 2^-21 (|a| + |b|) at most before it is rounded (the sine and cosine by 2^-23.2 of
1, of the products and their sum each by 2^-24).  A page's scale is that of the largest magnitude, so its exponent lies between
those of the largest less and plus delta: one value, but for a largest next to a border."""
import pytest
import torch

import exact_io_aware_52_b200 as fa
from exact_io_aware_52_b200 import _binding as fb
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


def dev():
    return torch.device("cuda:0")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def pair_sums(k, rot, layout):
    m = k.to(F64).abs()
    out = torch.zeros_like(m)
    if layout == "half":
        s = m[..., :rot // 2] + m[..., rot // 2:rot]
        out[..., :rot] = torch.cat([s, s], -1)
    else:
        out[..., :rot] = (m[..., 0:rot:2] + m[..., 1:rot:2]).repeat_interleave(2, -1)
    return out


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,N,H_kv,d,page,rot,start", [
    (2, 200, 3, 128, 128, 128, [0, 100]),   # 64 KB of sines
    (2, 130, 2, 256, 64, 256, [0, 37]),     # 64 KB
    (2, 300, 2, 256, 128, 256, [0, 90]),    # 128 KB, read twice
    (1, 128, 5, 256, 128, 128, [128]),      # 64 KB, read twice, half of a head turned
    (1, 1000, 1, 128, 128, 96, [5]),        # 48 KB
    (3, 1, 2, 256, 128, 256, [0, 127, 128]), (2, 4, 2, 128, 16, 128, [13, 16]),  # a warp each
    (1, 140, 2, 128, 128, 84, [60]),        # element by element
])
def test_turned_keys_at_full_width(layout, B, N, H_kv, d, page, rot, start):
    pool = ref.pool(90, [s + N for s in start], H_kv, page, d)
    g = torch.Generator().manual_seed(91)
    k, v = ((torch.randn(B, H_kv, N, d, generator=g) * torch.exp(torch.randn(B, H_kv, N, 1, generator=g))).to(BF16)
            for _ in range(2))
    kc, vc, ks, vs, table = (t.to(dev()) for t in pool)
    status = ints([0])
    fa.cache_append(fa.PagedCache(kc, vc, ks, vs, table), k.to(dev()), v.to(dev()), ints(start),
                    rotary=fa.Rotary(rot, layout=layout), dev_status=status)
    assert fa.read_device_status(status) == fb.FA_OK
    turned = ref.rope(k, torch.tensor(start)[:, None] + torch.arange(N), ref.angles(rot), layout)
    delta = pair_sums(k, rot, layout) * 2.0 ** -21
    codes, scales = kc.cpu().float().to(F64), ks.cpu().to(F64)
    before = pool[2].to(F64)
    seen = torch.zeros(pool[0].shape[0], dtype=torch.bool)
    borders = 0
    for b in range(B):
        t, end = start[b], start[b] + N
        while t < end:
            slot, p = t % page, int(pool[4][b, t // page])
            n = min(page - slot, end - t)
            seen[p] = True
            for h in range(H_kv):
                part = turned[b, h, t - start[b]:t - start[b] + n]
                err = delta[b, h, t - start[b]:t - start[b] + n]
                lo, hi = (2.0 ** ref.page_exponent(float((part.abs() + s * err).amax())) for s in (-1, 1))
                if slot:
                    lo, hi = max(lo, float(before[p, h])), max(hi, float(before[p, h]))
                s = float(scales[p, h])
                assert s in (lo, hi)
                borders += lo != hi
                got = codes[p, h, slot:slot + n] * s
                bound = torch.maximum(part.abs() * 2.0 ** -4, torch.full_like(part, s * 2.0 ** -10)) + err * (1 + 2.0 ** -4)
                assert ((got - part).abs() <= bound).all()
                if slot:  # the tokens from before, at the scale of now
                    want = ref.to_codes(pool[0].float().to(F64)[p, h, :slot] * (float(before[p, h]) / s))
                    assert torch.equal(codes[p, h, :slot], want)
            t += n
    assert borders <= 2  # of some dozen pages and heads, each next to a border with a chance of 2^-19
    assert torch.equal(kc.cpu().view(torch.uint8)[~seen], pool[0].view(torch.uint8)[~seen])
    assert torch.equal(ks.cpu()[~seen], pool[2][~seen])
    # the values, which are not turned, are exact
    wc, ws = pool[1].float().to(F64), pool[3].to(F64).clone()
    ref.append(wc, ws, pool[4], v.to(F64), start, [N] * B, page)
    assert torch.equal(vc.cpu().float().to(F64), wc) and torch.equal(vs.cpu().to(F64), ws)

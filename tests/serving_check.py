"""How far attention over the 8-bit cache may be from its definition in 64 bits, term by term, and
inputs in which every part of a split counts.  CPU only; nothing here imports the package.

Bounds, for a row with scores x_j, weights p_j (their sum 1), page scales ks, vs and codes k', v':

* score: q in fp16 is exact for these inputs, k' is exact, the products are exact in the
  tensor core, and each of the up to 16 + 3 sums of a chain is off by at most 2^-23 of the sum of the magnitudes; four
  factors by 2^-24: e_x = 2^-18 sum_i |q_i k_i| scale;
* weight: 2 e_x (numerator and sum), its rounding, and (|x| + |log2 vs| + 32) 2^-22 for
  the exponential, the logarithm of the scale and the references, which are numbers of that size in fp32.  The rounding is
  to two fp16 numbers (11 bits cut off, the rest below 2^-10 rounded by 2^-11 of itself: 2^-20 is above that), and to one, 2^-11,
  for bf16 outputs of more than 4 rows for each key;
* fp32 sums over the tiles of a warp, 16 tokens each and at most 512 of them, each off by 2^-23 (so is the sum of the
  weights), and over the lanes, the merge and its factors, less than 2^6 of them: 2^-17;
* a weight that is subnormal in fp16 errs by half of its step, 2^-25, where the row's largest p_j vs_j is at
  least 2^7: 2^-32 max_j (p_j vs_j) for each code;
* half a step of the output type, which below its smallest normal number 2^-126 is 2^-150 for fp32 (23 bits below
  it) and 2^-134 for bf16 (7 bits below it), and that of fp32 at each step of the merge: a part's O (1), the sums of
  at most 16 warps' and of at most 8 CTAs' parts, each of which is then divided by a sum of weights that is at least 1
  (the key that set the reference, or a larger one, has 1 or more), so by 24 at most in all, and the two quotients:
  less than 32 halves of a step, 2^-145.
"""
from __future__ import annotations

import math

import torch

from tests import serving_ref as ref

F64, BF16 = torch.float64, torch.bfloat16
STRIPE_SCALE = 2.0 ** -5  # scores of stripe_values' inputs spread by about 0.6: every block has a weight to be seen


def attend_terms(q, pool, lens, causal, scale, page):
    """O and lse of every row from the definition, and the bound's terms: sum_j p_j |v_j|, the largest
    sum_i |q_i k_i| * scale, max_j (p_j vs_j) and sum_j |v'_j|, and the largest |log2 vs|."""
    B, H, N, d = q.shape
    kc, vc, ks, vs, table = pool
    H_kv = kc.shape[1]
    ones = torch.ones_like(vs)
    o, oabs, codes = (torch.zeros(B, H, N, d, dtype=F64) for _ in range(3))
    lse, mag, top, log_vs = (torch.zeros(B, H, N, dtype=F64) for _ in range(4))
    lse.fill_(-math.inf)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k = ref.dense(kc.float(), ks, table.clamp(min=0), b, n, page)
        c = ref.dense(vc.float(), ones, table.clamp(min=0), b, n, page)
        s = vs[table[b, :-(-n // page)].clamp(min=0).long()].to(F64).t().repeat_interleave(page, 1)[:, :n]  # [H_kv, n]
        k, c, s = (t.repeat_interleave(H // H_kv, 0) for t in (k, c, s))
        for i in range(N):
            m = max(0, n - N + i + 1) if causal else n
            if m == 0:
                continue
            qi = q[b, :, i].to(F64)
            x = torch.einsum("hd,hnd->hn", qi, k[:, :m]) * scale
            lse[b, :, i] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            ps = p * s[:, :m]
            o[b, :, i] = torch.einsum("hn,hnd->hd", ps, c[:, :m])
            oabs[b, :, i] = torch.einsum("hn,hnd->hd", ps, c[:, :m].abs())
            codes[b, :, i] = c[:, :m].abs().sum(1)
            mag[b, :, i] = (torch.einsum("hd,hnd->hn", qi.abs(), k[:, :m].abs()) * scale).amax(-1)
            top[b, :, i] = ps.amax(-1)
            log_vs[b, :, i] = s[:, :m].clamp(min=2.0 ** -149).log2().abs().amax(-1)
    steps = torch.tensor([min(-(-n // 16), 512) for n in lens], dtype=F64)[:, None, None]
    return dict(o=o, lse=lse, oabs=oabs, codes=codes, mag=mag, top=top, log_vs=log_vs, steps=steps, rows=H // H_kv * N)


def bounds(t, dtype):
    """The bounds above for O (of that type) and lse."""
    e_x = t["mag"] * 2.0 ** -18
    weight = 2.0 ** -11 if dtype is BF16 and t["rows"] > 4 else 2.0 ** -20
    rel = 2 * e_x + weight + (1.5 * t["mag"] + t["log_vs"] + 32) * 2.0 ** -22 + 2 * t["steps"] * 2.0 ** -23 + 2.0 ** -17
    o = rel[..., None] * (t["oabs"] + t["o"].abs()) + t["codes"] * (2.0 ** -32 * t["top"])[..., None]
    o = o + (o + t["o"].abs()) * (2.0 ** -8 if dtype is BF16 else 2.0 ** -24) + 2.0 ** -145 + (2.0 ** -134 if dtype is BF16 else 0.0)
    return o, e_x + 2.0 ** -14 + 2.0 ** -22 * t["lse"].abs()


def off(o, lse, t):
    """The rows' first fault in words, or None."""
    bo, bl = bounds(t, o.dtype)
    got, gl = o.cpu().to(F64), lse.cpu().to(F64)
    empty = torch.isneginf(t["lse"])
    if not torch.equal(torch.isneginf(gl), empty) or not (got[empty] == 0).all():
        return "rows without keys"
    err = (got - t["o"]).abs()
    if not (err <= bo).all():
        return f"O: {float((err / bo).nan_to_num(math.inf).max())} times its bound"
    err = (gl - t["lse"]).abs()[~empty]
    if not (err <= bl[~empty]).all():
        return f"lse: off by {float(err.max())}"
    return None


def check(o, lse, q, pool, lens, causal, scale, page):
    fault = off(o, lse, attend_terms(q, pool, lens, causal, scale, page))
    assert fault is None, fault


def stripe_values(pool, lens, page, block):
    """Values under which no key can be left out unseen: token t has codes from 1 to 2 in the components that are
    t // block modulo d (plus half of d), and zeros elsewhere, and all pages have one scale: every component is a sum of
    positive terms of a few blocks."""
    kc, vc, ks, vs, table = pool
    d = kc.shape[3]
    vc, vs = torch.zeros_like(vc), torch.full_like(vs, 2.0 ** -5)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        at = table[b, t // page].long()
        c = (t // block) % d
        value = (1.0 + (t % 8) / 8.0).to(vc.dtype)[:, None].expand(n, kc.shape[1])
        for comp in (c, (c + d // 2) % d):
            vc.view(torch.uint8)[at, :, t % page, comp] = value.view(torch.uint8)
    return kc, vc, ks, vs, table

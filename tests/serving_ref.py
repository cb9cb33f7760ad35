"""Rotary positions and the paged 8-bit cache from their definitions in 64 bits on
the CPU (torch.float64), and the inputs of their tests.  Nothing here imports the
package."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
E4M3 = torch.float8_e4m3fn
MIN_EXP = -100


# ---------------------------------------------------------------- rotary positions
def angles(dim, base=10000.0, scaling="none", factor=1.0, original_length=0.0, low_turns=1.0, high_turns=32.0):
    """Radians per position of each pair."""
    if scaling == "base":
        base = base * factor ** (dim / (dim - 2))
    w = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        w = [x / factor for x in w]
    if scaling == "parts":
        out = []
        for x in w:
            keep = min(max((original_length * x / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0.0), 1.0)
            out.append(keep * x + (1.0 - keep) * x / factor)
        w = out
    return torch.tensor(w, dtype=F64)


def rope(x, pos, w, layout="half", inverse=False, amplitude=1.0):
    """x [B, heads, N, d] turned; pos [B, N]; w radians for each of the leading pairs."""
    x = x.to(F64)
    dim = 2 * len(w)
    ang = pos.to(F64)[:, None, :, None] * w
    c, s = ang.cos() * amplitude, ang.sin() * (-amplitude if inverse else amplitude)
    y = x.clone()
    ia = torch.arange(dim // 2) * (2 if layout == "interleaved" else 1)
    ib = ia + (1 if layout == "interleaved" else dim // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


# ---------------------------------------------------------------- the cache
def page_exponent(amax):
    """The least e >= MIN_EXP with amax <= 448 * 2^e."""
    e = MIN_EXP
    if amax > 448.0 * 2.0 ** MIN_EXP:
        e = math.ceil(math.log2(amax / 448.0))
        while amax > 448.0 * 2.0 ** e:
            e += 1
        while e > MIN_EXP and amax <= 448.0 * 2.0 ** (e - 1):
            e -= 1
    return e


def to_codes(x):
    """E4M3 rounding of values in range, from 64 bits (nearest, ties to even); NaN for what is not finite."""
    fin = torch.isfinite(x)
    y = torch.where(fin, x, torch.zeros_like(x))
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    r = (torch.round(a / step) * step).clamp(max=448.0) * torch.sign(y)  # torch.round: ties to even
    return torch.where(fin, r, torch.full_like(r, math.nan))


def append(codes, scales, table, x, start, n_new, page):
    """codes [P, H, page, d] and scales [P, H] in 64 bits, changed in place; x [B, H, N, d]."""
    B, H, N, d = x.shape
    for b in range(B):
        n = max(0, min(N, n_new[b]))
        t, end = start[b], start[b] + n
        while t < end:
            slot, p = t % page, int(table[b, t // page])
            m = min(page - slot, end - t)
            for h in range(H):
                part = x[b, h, t - start[b]:t - start[b] + m].to(F64)
                mag = part.abs()
                mag = mag[torch.isfinite(mag)]
                now = 2.0 ** page_exponent(float(mag.max()) if mag.numel() else 0.0)
                if slot:
                    old = float(scales[p, h])
                    now = max(now, old)
                    if now != old:
                        codes[p, h, :slot] = to_codes(codes[p, h, :slot] * (old / now))
                codes[p, h, slot:slot + m] = to_codes(part / now)
                scales[p, h] = now
            t += m


def dense(codes, scales, table, b, n, page, n_pages=None):
    """Values of the first n tokens of sequence b, [H, n, d] in 64 bits."""
    need = -(-n // page)
    p = table[b, :need].long()
    x = codes[p].to(F64) * scales[p].to(F64)[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :n]


def attend(q, k, v, lens, causal, scale):
    """q [B, H, N, d]; k, v: for each sequence [H_kv, n, d] in 64 bits.  Returns O, lse, and for the
    error bounds sum_j p_j |v_j| and the largest sum_i |q_i k_i| * scale of each row."""
    B, H, N, d = q.shape
    o = torch.zeros(B, H, N, d, dtype=F64)
    lse = torch.full((B, H, N), -math.inf, dtype=F64)
    oabs = torch.zeros_like(o)
    mag = torch.zeros_like(lse)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        g = H // k[b].shape[0]
        for i in range(N):
            m = max(0, n - N + i + 1) if causal else n
            if m == 0:
                continue
            kk = k[b][:, :m].repeat_interleave(g, 0)
            vv = v[b][:, :m].repeat_interleave(g, 0)
            qq = q[b, :, i].to(F64)
            x = torch.einsum("hd,hnd->hn", qq, kk) * scale
            mag[b, :, i] = (torch.einsum("hd,hnd->hn", qq.abs(), kk.abs()) * scale).amax(-1)
            lse[b, :, i] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            o[b, :, i] = torch.einsum("hn,hnd->hd", p, vv)
            oabs[b, :, i] = torch.einsum("hn,hnd->hd", p, vv.abs())
    return o, lse, oabs, mag


# ---------------------------------------------------------------- inputs
def pool(seed, lens, H_kv, page, d, extra=3, spread=(-8, -3)):
    """A pool of random codes with power-of-two scales, and a table with the pages in random order
    (-1 behind a sequence's last)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    shape = (n_pages, H_kv, page, d)
    kc, vc = ((torch.randn(shape, generator=g) * 80.0).clamp(-448, 448).to(E4M3) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(spread[0], spread[1], shape[:2], generator=g).float()) for _ in range(2))
    return kc, vc, ks, vs, table

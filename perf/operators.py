"""The cases of the rotary positions and of the 8-bit paged key/value cache.

Four operators that one serving or training step uses together:

* ``rope``    rotary positions of queries and keys, or their inverse for gradients;
* ``append``  new keys (rotated on the way) and values written into a paged E4M3 cache
  with one power-of-two scale for each (page, key/value head);
* ``attend``  attention of a few query tokens for each sequence over that cache;
* ``gather``  the cache as contiguous bfloat16 keys and values.

With ``own`` false they are computed in elementary torch operations, with ``own``
true by this repository's package.  ``exact`` has each from its definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
MIN_EXP = -100  # smallest exponent of a page's scale


# ---------------------------------------------------------------- the cases
def _rope(name, B, N, H, Hkv, d, rot, layout="half", scaling="none", factor=1.0, inverse=False, src="bf16",
          far=0, strided=False):
    return dict(name=name, op="rope", B=B, N=N, H=H, Hkv=Hkv, d=d, rot=rot, layout=layout, scaling=scaling,
                factor=factor, inverse=inverse, src=src, far=far, strided=strided)


def _append(name, B, N, Hkv, d, page, lo, hi, rot=0, layout="half", ragged=False):
    return dict(name=name, op="append", B=B, N=N, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, rot=rot, layout=layout,
                ragged=ragged)


def _attend(name, B, N, H, Hkv, d, page, lo, hi, causal=True):
    return dict(name=name, op="attend", B=B, N=N, H=H, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, causal=causal)


def _gather(name, B, Hkv, d, page, lo, hi):
    return dict(name=name, op="gather", B=B, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi)


def listed():
    return [
        # one new token for each of four sequences deep in a long context: latency
        _rope("rope one token", 4, 1, 32, 8, 128, 128, scaling="parts", factor=8.0, far=100_000),
        # the queries and keys of a training step, read out of a fused projection's [B, N, heads, d]
        _rope("rope training", 2, 8192, 32, 8, 128, 128, strided=True),
        # the gradients that the backward pass leaves in fp32, rotated back; half of each head, an odd length
        _rope("rope gradient", 2, 4097, 16, 16, 128, 64, layout="interleaved", inverse=True, src="f32"),
        # decoding: one token for each of 64 sequences, most of them in the middle of a page
        _append("append one token", 64, 1, 8, 128, 64, 0, 255, rot=128),
        # four prompts of different lengths, onto sequences that hold some tokens already
        _append("append prompts", 4, 8192, 8, 128, 64, 0, 100, rot=128, ragged=True),
        # short odd chunks, small pages, narrow heads, keys that come rotated
        _append("append chunks", 16, 777, 12, 64, 16, 1, 333),
        # one short sequence: latency
        _attend("attend one short", 1, 1, 32, 8, 128, 64, 500, 500),
        # a batch of ragged sequences, one token each
        _attend("attend batch", 64, 1, 32, 8, 128, 64, 1, 8192),
        # long contexts with grouped heads
        _attend("attend long", 8, 1, 32, 8, 128, 128, 16_384, 131_072),
        # five drafted tokens for each sequence, every head its own keys, small pages
        _attend("attend drafts", 8, 5, 12, 12, 64, 16, 700, 9000),
        # a cached prefix handed to the prompt's attention
        _gather("gather short", 1, 8, 128, 64, 1000, 1000),
        _gather("gather long", 4, 8, 128, 64, 9000, 32_768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "gather"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    page = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        H = Hkv * rng.choice([1, 2, 4])
        tokens = max(1, min(200_000_000 // (2 * d * (H + Hkv) * 2), _log(rng, 1, 20_000)))
        B = _log(rng, 1, min(64, tokens))
        scaling = rng.choice(["none", "linear", "base", "parts"])
        rot = rng.choice([d, d // 2, d // 4])
        inverse = rng.random() < 0.4
        return _rope("", B, max(1, tokens // B), H, Hkv, d, rot, layout, scaling, 1.0 if scaling == "none" else
                     rng.choice([2.0, 8.0, 20.0]), inverse, "f32" if inverse else "bf16", _log(rng, 1, 1_000_000),
                     rng.random() < 0.5)
    if op == "append":
        B = _log(rng, 1, 64)
        N = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, min(8192, 40_000_000 // (d * Hkv * B))))
        return _append("", B, N, Hkv, d, page, 0, _log(rng, 1, 400), rng.choice([0, d, d // 2]), layout,
                       N > 1 and rng.random() < 0.5)
    most = 400_000_000 // (d * Hkv)  # tokens over all sequences
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, max(1, min(131_072, most // B)))
    lo = rng.choice([0, 1, hi // 2, hi]) if hi > 1 else 1
    if op == "attend":
        return _attend("", B, rng.choice([1, 1, 1, 2, 3, 4, 7]), Hkv * rng.choice([1, 2, 4, 8]), Hkv, d, page, lo, hi,
                       rng.random() < 0.8)
    hi = min(hi, max(1, 100_000_000 // (d * Hkv * B)))
    return _gather("", B, Hkv, d, page, min(lo, hi), hi)


def _lengths(c):
    """Tokens that each sequence's cache holds before the call."""
    r = random.Random(c["B"] * 1_000_003 + c["hi"])
    n = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    n[r.randrange(c["B"])] = c["hi"]
    return n


def _new_tokens(c):
    """Tokens that each sequence appends."""
    r = random.Random(c["B"] * 7_919 + c["N"])
    return [r.randint(0, c["N"]) if c["ragged"] and b else c["N"] for b in range(c["B"])]


def work(c):
    op, d = c["op"], c["d"]
    if op == "rope":
        n = c["B"] * c["N"] * (c["H"] + c["Hkv"])
        return {"bytes": n * d * (6 if c["src"] == "f32" else 4) + 4 * c["B"] * c["N"], "flops": 3 * n * c["rot"]}
    if op == "append":
        n = sum(_new_tokens(c)) * c["Hkv"]
        pages = sum(-(-(s + a) // c["page"]) - s // c["page"] for s, a in zip(_lengths(c), _new_tokens(c)) if a)
        return {"bytes": 6 * n * d + pages * (8 * c["Hkv"] + 4) + 8 * c["B"], "flops": n * (3 * c["rot"] + 4 * d)}
    n = sum(_lengths(c)) * c["Hkv"]
    pages = sum(-(-s // c["page"]) for s in _lengths(c))
    side = pages * (8 * c["Hkv"] + 4) + 4 * c["B"]
    if op == "attend":
        rows = c["B"] * c["H"] * c["N"]
        group = c["H"] // c["Hkv"]
        return {"bytes": 2 * n * d + side + rows * (4 * d + 4), "flops": 4 * n * group * c["N"] * d}
    return {"bytes": 2 * n * d + side + 4 * c["B"] * c["Hkv"] * c["hi"] * d, "flops": 2 * n * d}


# ---------------------------------------------------------------- the inputs
def _codes(gen, shape):
    """E4M3 codes of normally distributed values that fill a page's range."""
    out = torch.empty(shape, dtype=E4M3, device=DEV)
    for i in range(0, shape[0], 1024):
        part = torch.randn(out[i:i + 1024].shape, generator=gen, device=DEV)
        out[i:i + 1024] = (part * 80.0).clamp_(-448.0, 448.0).to(E4M3)
    return out


def _pool(c, gen, seed, total):
    """The cache: codes, scales and a page table whose pages lie in random order."""
    need = [-(-t // c["page"]) for t in total]
    n_pages = sum(need) + 3
    order = list(range(n_pages))
    random.Random(seed).shuffle(order)
    table = torch.full((c["B"], max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    shape = (n_pages, c["Hkv"], c["page"], c["d"])
    scales = [torch.exp2(torch.randint(-8, -4, shape[:2], generator=gen, device=DEV).float()) for _ in range(2)]
    return dict(kc=_codes(gen, shape), vc=_codes(gen, shape), ks=scales[0], vs=scales[1], table=table.to(DEV))


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=c)
    B, d = c["B"], c["d"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    if c["op"] == "rope":
        dt = F32 if c["src"] == "f32" else BF16
        heads, N = c["H"] + c["Hkv"], c["N"]
        if c["strided"]:
            x = randn(B, N, heads, d).to(dt).transpose(1, 2)
            s["q"], s["k"] = x[:, :c["H"]], x[:, c["H"]:]
        else:
            s["q"], s["k"] = randn(B, c["H"], N, d).to(dt), randn(B, c["Hkv"], N, d).to(dt)
        first = torch.randint(0, max(1, c["far"]) + 1, (B, 1), generator=gen, device=DEV)
        s["pos"] = (first + torch.arange(N, device=DEV)).to(torch.int32)
        return s
    held = _lengths(c)
    if c["op"] == "append":
        new = _new_tokens(c)
        s |= _pool(c, gen, seed, [a + b for a, b in zip(held, new)])
        # keys and values as a fused projection leaves them, [B, N, 2, heads, d], a spread that differs by token
        x = randn(B, c["N"], 2, c["Hkv"], d) * torch.exp(0.5 * randn(B, c["N"], 1, 1, 1))
        x = x.to(BF16)
        s["k"], s["v"] = x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2)
        s["start"] = torch.tensor(held, dtype=torch.int32, device=DEV)
        s["new"] = torch.tensor(new, dtype=torch.int32, device=DEV)
        return s
    s |= _pool(c, gen, seed, held)
    s["len"] = torch.tensor(held, dtype=torch.int32, device=DEV)
    if c["op"] == "attend":
        s["q"] = randn(B, c["H"], c["N"], d).to(BF16)
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ---------------------------------------------------------------- the plain forms
def _angles(c):
    """Radians by which each pair of a head turns from one position to the next, in 64 bits."""
    r = c["rot"]
    base, factor, kind = 10000.0, c.get("factor", 1.0), c.get("scaling", "none")
    if kind == "base":
        base = base * factor ** (r / (r - 2))
    a = base ** (-torch.arange(0, r, 2, dtype=F64, device=DEV) / r)
    if kind == "linear":
        a = a / factor
    if kind == "parts":  # few turns within 4096 positions: stretched by `factor`; many: left
        mix = ((4096.0 * a / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        a = a * (mix + (1.0 - mix) / factor)
    return a


def _turned(x, cos, sin, rot, layout):
    """x [..., d] with its first `rot` components turned, pair by pair."""
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([head, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    ang = s["pos"].to(F64)[:, None, :, None] * _angles(c)
    cos, sin = ang.cos().to(F32), ang.sin().to(F32)
    sin = -sin if c["inverse"] else sin
    return [_turned(s[t].to(F32), cos, sin, c["rot"], c["layout"]).to(BF16) for t in ("q", "k")]


def _scale_of(amax):
    """The smallest power of two by which `amax` reaches no further than 448."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_append(s):
    c = s["case"]
    B, N, Hkv, page = c["B"], c["N"], c["Hkv"], c["page"]
    start, new = s["start"].long(), s["new"].long()
    at = start[:, None] + torch.arange(N, device=DEV)  # [B, N] position of each token
    live = torch.arange(N, device=DEV) < new[:, None]
    k = s["k"].to(F32)
    if c["rot"]:
        ang = at.to(F64)[:, None, :, None] * _angles(c)
        k = _turned(k, ang.cos().to(F32), ang.sin().to(F32), c["rot"], c["layout"])
    b, i = live.nonzero(as_tuple=True)
    phys = s["table"].long()[b, at[b, i] // page]
    slot = at[b, i] % page
    # pages that hold tokens from before: one at most for each sequence
    part = ((start % page > 0) & (new > 0)).nonzero(as_tuple=True)[0]
    old_page = s["table"].long()[part, start[part] // page]
    keep = (torch.arange(page, device=DEV) < (start[part] % page)[:, None])[:, None, :, None]
    for x, codes, scales in ((k, s["kc"], s["ks"]), (s["v"].to(F32), s["vc"], s["vs"])):
        x = x[b, :, i]  # [tokens, Hkv, d]
        amax = torch.zeros_like(scales).index_reduce_(0, phys, x.abs().amax(-1), "amax")
        now = _scale_of(amax)
        now[old_page] = torch.maximum(now[old_page], scales[old_page])
        old = codes[old_page].to(F32) * (scales[old_page] / now[old_page])[..., None, None]
        old = torch.where(keep, old.to(E4M3).to(F32), codes[old_page].to(F32)).to(E4M3)
        codes.view(torch.uint8)[old_page] = old.view(torch.uint8)
        codes.view(torch.uint8)[phys, :, slot] = (x / now[phys][..., None]).to(E4M3).view(torch.uint8)
        scales[phys] = now[phys]
    return [s["kc"], s["ks"], s["vc"], s["vs"]]


def _dense(s, codes, scales):
    """The cache's values, [B, Hkv, tokens, d] in 32 bits, zero behind each sequence's end."""
    c = s["case"]
    t = s["table"].long().clamp(min=0)
    x = codes.view(torch.uint8)[t].view(E4M3).to(F32) * scales[t][..., None, None]  # [B, pages, Hkv, page, d]
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :max(1, c["hi"])]
    live = torch.arange(x.shape[2], device=DEV) < s["len"][:, None]
    return torch.where(live[:, None, :, None], x, 0.0), live


def _plain_attend(s):
    c = s["case"]
    B, N, Hkv, d = c["B"], c["N"], c["Hkv"], c["d"]
    k, live = _dense(s, s["kc"], s["ks"])
    q = s["q"].to(F32).view(B, Hkv, -1, d)
    x = (q @ k.transpose(2, 3)).view(B, Hkv, -1, N, k.shape[2]) * s["scale"]
    del k
    ok = live[:, None, None, None, :]
    if c["causal"]:
        last = s["len"][:, None] - N + torch.arange(N, device=DEV)  # position of each query
        ok = ok & (torch.arange(x.shape[-1], device=DEV) <= last[:, :, None])[:, None, None]
    x = torch.where(ok, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).view(B, c["H"], N)
    p = p / torch.where(total > 0, total, 1.0)
    v, _ = _dense(s, s["vc"], s["vs"])
    o = p.view(B, Hkv, -1, v.shape[2]) @ v
    return [o.view(B, c["H"], N, d).to(BF16), lse]


def _plain_gather(s):
    return [_dense(s, s[x + "c"], s[x + "s"])[0].to(BF16) for x in ("k", "v")]


# ---------------------------------------------------------------- one pass
def _rotary(fa, c):
    if not c["rot"]:
        return None
    return fa.Rotary(c["rot"], layout=c["layout"], base=10000.0, scaling=c.get("scaling", "none"),
                     factor=c.get("factor", 1.0), original_length=4096, low_turns=1.0, high_turns=32.0)


def _handles(s):
    """What a program that uses the package keeps beside its tensors: the rotation's table and the cache's handle."""
    if "handles" not in s:
        import exact_io_aware_52_b200 as fa
        c = s["case"]
        s["handles"] = (fa, _rotary(fa, c) if "rot" in c else None,
                        None if c["op"] == "rope" else fa.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"], s["table"]))
    return s["handles"]


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "gather": _plain_gather}[c["op"]](s)
    fa, rotary, cache = _handles(s)
    if c["op"] == "rope":
        return list(fa.rope(rotary, s["q"], s["k"], pos=s["pos"], inverse=c["inverse"], out_dtype=BF16))
    if c["op"] == "append":
        fa.cache_append(cache, s["k"], s["v"], s["start"], n_new=s["new"], rotary=rotary)
        return [s["kc"], s["ks"], s["vc"], s["vs"]]
    if c["op"] == "attend":
        return list(fa.cache_attention(cache, s["q"], s["len"], c["causal"], s["scale"], out_dtype=BF16))
    return list(fa.cache_gather(cache, s["len"], max(1, c["hi"])))


# ---------------------------------------------------------------- 64 bits
def _exact_turn(x, pos, c, sign):
    """Each pair as a complex number times exp(i position angle)."""
    r = c["rot"]
    n = torch.arange(r // 2, dtype=F64, device=DEV)
    factor, kind = c.get("factor", 1.0), c.get("scaling", "none")
    logbase = math.log(10000.0) + (math.log(factor) * r / (r - 2) if kind == "base" else 0.0)
    w = torch.exp(-2.0 * n / r * logbase)
    if kind == "linear":
        w = w / factor
    if kind == "parts":
        keep = torch.clamp((4096.0 * w / math.tau - 1.0) / 31.0, min=0.0, max=1.0)
        w = keep * w + (1.0 - keep) * w / factor
    one = torch.polar(torch.ones((), dtype=F64, device=DEV), sign * pos.to(F64)[..., None] * w)  # [B, N, r/2]
    first = torch.arange(r // 2, device=DEV) * (1 if c["layout"] == "half" else 2)
    second = first + (r // 2 if c["layout"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * one[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append(s):
    c, out = s["case"], []
    held, new = _lengths(c), _new_tokens(c)
    pos = s["start"].long()[:, None] + torch.arange(c["N"], device=DEV)
    for name in "kv":
        x = s[name].to(F64)
        if name == "k" and c["rot"]:
            x = _exact_turn(x, pos, c, 1.0)
        codes, scales = s[name + "c"].to(F64), s[name + "s"].to(F64)
        for b in range(c["B"]):
            t, end = held[b], held[b] + new[b]
            while t < end:
                slot, p = t % c["page"], int(s["table"][b, t // c["page"]])
                n = min(c["page"] - slot, end - t)
                part = x[b, :, t - held[b]:t - held[b] + n]
                most = part.abs().amax((1, 2))
                e = torch.ceil(torch.log2(most / 448.0)).clamp(min=MIN_EXP)
                e = e - (most <= 448.0 * torch.exp2(e - 1.0)).to(F64)  # a logarithm rounded up over its border
                now = torch.exp2(e.clamp(min=MIN_EXP))
                if slot:
                    now = torch.maximum(now, scales[p])
                    codes[p, :, :slot] = (codes[p, :, :slot] * (scales[p] / now)[:, None, None]).to(F32).to(E4M3).to(F64)
                codes[p, :, slot:slot + n] = (part / now[:, None, None]).to(F32).to(E4M3).to(F64)
                scales[p] = now
                t += n
        out += [codes, scales]
    return out


def _exact_rows(s, name, b):
    c, n = s["case"], _lengths(s["case"])[b]
    p = s["table"][b, :-(-n // c["page"])].long()
    x = s[name + "c"].view(torch.uint8)[p].view(E4M3).to(F64) * s[name + "s"][p].to(F64)[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(c["Hkv"], -1, c["d"])[:, :n]


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return [_exact_turn(s[t].to(F64), s["pos"], c, -1.0 if c["inverse"] else 1.0) for t in ("q", "k")]
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "gather":
        out = [torch.zeros(c["B"], c["Hkv"], max(1, c["hi"]), c["d"], dtype=F64, device=DEV) for _ in "kv"]
        for o, name in zip(out, "kv"):
            for b, n in enumerate(_lengths(c)):
                o[b, :, :n] = _exact_rows(s, name, b)
        return out
    B, N, H, d = c["B"], c["N"], c["H"], c["d"]
    o = torch.zeros(B, H, N, d, dtype=F64, device=DEV)
    lse = torch.full((B, H, N), -math.inf, dtype=F64, device=DEV)
    for b, n in enumerate(_lengths(c)):
        if not n:
            continue
        k, v = _exact_rows(s, "k", b), _exact_rows(s, "v", b)
        for i in range(N):
            m = max(0, n - N + i + 1) if c["causal"] else n
            if not m:
                continue
            q = s["q"][b, :, i].to(F64).view(c["Hkv"], -1, d)
            x = torch.einsum("hgd,hnd->hgn", q, k[:, :m]) * s["scale"]
            lse[b, :, i] = torch.logsumexp(x, -1).view(H)
            o[b, :, i] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v[:, :m]).reshape(H, d)
    return [o, lse]

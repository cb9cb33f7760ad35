"""Rotary positions and the paged 8-bit cache on the GPU against their definitions in
64 bits (serving_ref).

Bounds.  u = 2^-24 is half a step of fp32.
* rope: the angle's float and sincospi err by 2^-25 pi and 2 u, the two products and
  their sum by 3 u each: at most 2^-21 (|a| + |b|) * amplitude; then half a step of the output (2^-8 |y| for
  bf16).
* cache_append: without rotation scales and codes are equal.  With it a value errs by the
  above before it is rounded: half a step of E4M3 (2^-4 relative, 2^-10 of the scale for subnormal codes)
  and that.
* cache_attention: a score (in units of ln) errs by e_x = 2^-21 sum |q k| scale, the fp32 sums of up to 272
  products and the factors; a weight by 2 e_x + 2^-11 (fp16) + 2^-18 (exponential, logarithm of the
  scale, fp32 sums, merges), or, if it is far below the row's largest, by 2^-31 of that.  So O errs by
  (2 e_x + 2^-11 + 2^-18) * (sum_j p_j |v_j| + |O|) + n 2^-31 max_j (p_j vs_j) 448, and half a step of the output; lse by
  e_x + 2^-18 + 2^-23 |lse|.
* cache_gather: equal (power-of-two scales).
"""
import math

import pytest
import torch

import exact_io_aware_52_b200 as fa
from exact_io_aware_52_b200 import _binding as fb
from tests import serving_ref as ref
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def dev():
    return torch.device("cuda:0")


# ---------------------------------------------------------------- rope
def check_rope(y, x, pos, rot_kw, dim, inverse=False, amplitude=1.0):
    layout = rot_kw.get("layout", "half")
    w = ref.angles(dim, **{k: v for k, v in rot_kw.items() if k != "layout"})
    want = ref.rope(x.cpu(), pos.cpu(), w, layout, inverse, amplitude)
    mag = x.cpu().to(F64).abs()
    pair = mag.clone()
    if layout == "half":
        s = mag[..., :dim // 2] + mag[..., dim // 2:dim]
        pair[..., :dim] = torch.cat([s, s], -1)
    else:
        pair[..., :dim] = (mag[..., 0:dim:2] + mag[..., 1:dim:2]).repeat_interleave(2, -1)
    pair[..., dim:] = 0.0
    err = (y.cpu().to(F64) - want).abs()
    bound = pair * (2.0 ** -21 * amplitude) + want.abs() * (2.0 ** -8 if y.dtype == BF16 else 2.0 ** -24)
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hkv,N,d,dim", [
    (1, 1, 1, 1, 64, 64), (2, 8, 2, 33, 128, 128), (3, 5, 1, 257, 128, 64), (1, 4, 4, 65, 256, 256), (2, 3, 3, 7, 80, 80),
    (1, 2, 2, 9, 64, 16), (2, 2, 1, 5, 96, 50), (1, 3, 1, 4, 33, 6), (1, 1, 1, 300, 1024, 256), (4, 1, 1, 2, 2, 2)])
@pytest.mark.parametrize("src,dst", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_rope_shapes(layout, B, H, Hkv, N, d, dim, src, dst):
    g = torch.Generator().manual_seed(d * 7 + N)
    q = torch.randn(B, H, N, d, generator=g).to(src).to(dev())
    k = torch.randn(B, Hkv, N, d, generator=g).to(src).to(dev())
    pos = torch.randint(0, 100_000, (B, N), generator=g, dtype=torch.int32)
    r = fa.Rotary(dim, layout=layout)
    yq, yk = fa.rope(r, q, k, pos=pos.to(dev()), out_dtype=dst)
    check_rope(yq, q, pos, dict(layout=layout), dim)
    check_rope(yk, k, pos, dict(layout=layout), dim)
    zq = fa.rope(r, q, pos=pos.to(dev()), inverse=True, out_dtype=dst)
    check_rope(zq, q, pos, dict(layout=layout), dim, inverse=True)


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0), dict(base=5e5),
                                dict(scaling="parts", factor=20.0, original_length=4096.0, low_turns=1.0, high_turns=32.0)])
def test_rope_long_contexts_and_far_positions(kw):
    g = torch.Generator().manual_seed(3)
    q = torch.randn(2, 4, 64, 128, generator=g).to(dev())
    pos = torch.randint(0, 2 ** 23, (2, 64), generator=g, dtype=torch.int32)
    pos[0, 0], pos[1, 5], pos[1, 6] = 2 ** 31 - 1, -1, -(2 ** 31)
    y = fa.rope(fa.Rotary(128, amplitude=1.25, **kw), q, pos=pos.to(dev()))
    # the reference's own angle in 64 bits errs by |pos| * 2^-53 at most: 2^-22 at the farthest
    keep = pos.abs() < 2 ** 26
    for b in range(2):
        n = keep[b].nonzero().flatten()
        check_rope(y[b:b + 1, :, n.to(dev())], q[b:b + 1, :, n.to(dev())], pos[b:b + 1, n], kw, 128, amplitude=1.25)
    assert torch.isfinite(y).all()


def test_rope_far_position_is_exact():
    """At 2^31 - 1 with one turn in 2^-k of a turn the angle is known exactly."""
    r = fa.Rotary(4, angles=[2 * math.pi / 8, 2 * math.pi * 3 / 16])
    for i in range(2):  # the steps are off by the rounding of the angles' doubles
        assert abs(r.struct.step[i] - (1 << 64) * (1 / 8, 3 / 16)[i]) <= 2 ** 13
    q = torch.zeros(1, 1, 1, 4, device=dev())
    q[..., :2] = 1.0
    p = 2 ** 31 - 1
    y = fa.rope(r, q, pos=torch.tensor([[p]], dtype=torch.int32, device=dev())).flatten().cpu().double()
    for i, turn in enumerate((p / 8 % 1, 3 * p / 16 % 1)):
        assert abs(y[i] - math.cos(2 * math.pi * turn)) <= 2.0 ** -18 and abs(y[i + 2] - math.sin(2 * math.pi * turn)) <= 2.0 ** -18


@pytest.mark.parametrize("how", ["transposed", "projection", "slice", "odd", "expanded"])
def test_rope_strides(how):
    g = torch.Generator().manual_seed(11)
    B, H, N, d = 2, 6, 19, 128
    if how == "transposed":
        x = torch.randn(B, N, H, d, generator=g).to(BF16).to(dev()).transpose(1, 2)
    elif how == "projection":
        x = torch.randn(B, N, 3, H, d, generator=g).to(BF16).to(dev())[:, :, 1].transpose(1, 2)
    elif how == "slice":
        x = torch.randn(B, H, 2 * N, d + 64, generator=g).to(BF16).to(dev())[:, :, ::2, 32:32 + d]
    elif how == "odd":
        x = torch.randn(B, H, N, d + 3, generator=g).to(BF16).to(dev())[..., 1:1 + d]
    else:
        x = torch.randn(B, 1, N, d, generator=g).to(BF16).to(dev()).expand(B, H, N, d)
    pos = torch.randint(0, 5000, (N,), generator=g, dtype=torch.int32)
    r = fa.Rotary(64, layout="interleaved")
    y = fa.rope(r, x, pos=pos.to(dev()))
    check_rope(y, x, pos.expand(B, N), dict(layout="interleaved"), 64)
    # into an output with strides of its own, the components around it left as they are
    big = torch.full((B, N, H, d + 16), 7.0, dtype=F32, device=dev())
    out = big[..., 8:8 + d].transpose(1, 2)
    assert fa.rope(r, x, pos0=40, out=out) is out
    check_rope(out, x, (torch.arange(N) + 40).expand(B, N), dict(layout="interleaved"), 64)
    assert (big[..., :8] == 7).all() and (big[..., 8 + d:] == 7).all()


@pytest.mark.parametrize("d,dim", [(128, 128), (128, 32), (72, 20)])
def test_rope_in_place(d, dim):
    g = torch.Generator().manual_seed(12)
    x = torch.randn(2, 3, 40, 4, d, generator=g).to(BF16).to(dev())
    q, k = x[:, 0].transpose(1, 2), x[:, 1].transpose(1, 2)
    keep, rest = x.clone(), x[:, 2].clone()
    r = fa.Rotary(dim)
    fa.rope(r, q, k, out=(q, k), pos0=100)
    pos = (torch.arange(40) + 100).expand(2, 40)
    check_rope(q, keep[:, 0].transpose(1, 2), pos, {}, dim)
    check_rope(k, keep[:, 1].transpose(1, 2), pos, {}, dim)
    assert torch.equal(x[:, 2], rest)
    # one in place, the other not
    q2, k2 = q.clone(), k.clone()
    yk = torch.zeros_like(k2)
    fa.rope(r, q2, k2, out=(q2, yk), pos0=3, inverse=True)
    check_rope(yk, k2, (torch.arange(40) + 3).expand(2, 40), {}, dim, inverse=True)
    check_rope(q2, q, (torch.arange(40) + 3).expand(2, 40), {}, dim, inverse=True)


def test_rope_writes_within_its_output_and_empty():
    g = torch.Generator().manual_seed(13)
    for d, N in ((128, 37), (50, 3)):
        q = torch.randn(2, 3, N, d, generator=g).to(BF16).to(dev())
        o = Guarded((2, 3, N, d), BF16, dev(), fill=float("nan"))
        fa.rope(fa.Rotary(d), q, out=o.t)
        o.check("rope")
        assert torch.isfinite(o.t).all()
    assert fa.rope(fa.Rotary(64), torch.empty(2, 0, 5, 64, device=dev())).shape == (2, 0, 5, 64)
    assert fa.rope(fa.Rotary(64), torch.empty(2, 3, 0, 64, device=dev())).shape == (2, 3, 0, 64)


def test_rope_gradient_through_attention():
    """dQ of softmax((R q)(R k)^T) v against the 64-bit formula: the backward pass's gradients
    turned back."""
    g = torch.Generator().manual_seed(14)
    B, H, Hkv, N, d = 1, 4, 2, 160, 64
    scale = d ** -0.5
    q, k, v, do = (torch.randn(B, h, N, d, generator=g).to(BF16) for h in (H, Hkv, Hkv, H))
    r = fa.Rotary(d)
    rq, rk = fa.rope(r, q.to(dev()), k.to(dev()))
    vd = v.to(dev())
    o, lse = fa.attention(rq, rk, vd, True, scale)
    dq, dk, dv = fa.attention_bwd(rq, rk, vd, o, lse, do.to(dev()), True, scale)
    gq, gk = fa.rope(r, dq, dk, inverse=True)
    w, pos = ref.angles(d), torch.arange(N).expand(B, N)
    q6, k6, v6 = (t.to(F64).requires_grad_() for t in (q, k, v))
    a = ref.rope(q6, pos, w)
    b = ref.rope(k6, pos, w).repeat_interleave(H // Hkv, 1)
    x = (a @ b.transpose(2, 3)) * scale
    x = x.masked_fill(torch.ones(N, N).triu(1).bool(), -math.inf)
    (torch.softmax(x, -1) @ v6.repeat_interleave(H // Hkv, 1)).backward(do.to(F64))
    for got, want in ((gq, q6.grad), (gk, k6.grad), (dv, v6.grad)):
        err = (got.cpu().to(F64) - want).norm() / want.norm()
        # P and dS are rounded to bf16 (2^-8 each), the turned q and k as well: each at most once in a
        # product, errors of random sign add as squares: 2^-8 * sqrt(4)
        assert err <= 2.0 ** -7, float(err)


# ---------------------------------------------------------------- the cache
def to_gpu(pool):
    return tuple(t.to(dev()) for t in pool)


def cache_of(pool):
    return fa.PagedCache(*to_gpu(pool))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


def as64(codes):
    return codes.cpu().to(F32).to(F64)


APPEND_SHAPES = [  # B, N, H_kv, d, page, start, n_new
    (1, 1, 1, 64, 16, [0], None), (3, 1, 2, 128, 64, [63, 64, 65], None), (2, 5, 3, 128, 16, [14, 31], [5, 2]),
    (2, 200, 2, 64, 32, [0, 31], [200, 0]), (2, 130, 1, 256, 128, [100, 0], [130, 129]), (4, 33, 2, 128, 128, [0, 1, 127, 128], None),
    (2, 64, 1, 256, 64, [64, 10], [70, -3]), (1, 300, 2, 256, 16, [7], None), (2, 17, 4, 64, 128, [120, 0], None),
]


def run_append(seed, B, N, H_kv, d, page, start, n_new, rot=None, layout="half", grow=1.0, x_of=None, offset=0):
    g = torch.Generator().manual_seed(seed)
    n = [max(0, min(N, a)) for a in (n_new or [N] * B)]
    pool = ref.pool(seed, [s + a for s, a in zip(start, n)], H_kv, page, d)
    x = torch.randn(B, N, 2, H_kv, d + offset, generator=g) * torch.exp(torch.randn(B, N, 1, 1, 1, generator=g)) * grow
    x = x.to(BF16)
    if x_of is not None:
        x_of(x)
    k, v = (x[:, :, i, :, offset:].transpose(1, 2) for i in (0, 1))
    xd = x.to(dev())
    kd, vd = (xd[:, :, i, :, offset:].transpose(1, 2) for i in (0, 1))
    dpool = to_gpu(pool)
    status = ints([0])
    fa.cache_append(fa.PagedCache(*dpool), kd, vd, ints(start), n_new=None if n_new is None else ints(n_new),
                    rotary=None if rot is None else fa.Rotary(rot, layout=layout), dev_status=status)
    assert fa.read_device_status(status) == fb.FA_OK
    return pool, dpool, k, v, n


@pytest.mark.parametrize("shape", APPEND_SHAPES)
@pytest.mark.parametrize("grow,offset", [(1.0, 0), (1e-3, 0), (100.0, 0), (1.0, 1)])
def test_append_is_exact(shape, grow, offset):
    B, N, H_kv, d, page, start, n_new = shape
    pool, dpool, k, v, n = run_append(17, *shape, grow=grow, offset=offset)
    for codes, scales, x, gc, gs in ((pool[0], pool[2], k, dpool[0], dpool[2]), (pool[1], pool[3], v, dpool[1], dpool[3])):
        wc, ws = as64(codes), scales.to(F64).clone()
        ref.append(wc, ws, pool[4], x.to(F64), start, n, page)
        assert torch.equal(gs.cpu().to(F64), ws)
        assert torch.equal(as64(gc), wc)  # pages that are not touched and slots behind the end among them


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [16, 64, 50])
@pytest.mark.parametrize("shape", APPEND_SHAPES[1:5])
def test_append_turns_keys(layout, rot, shape):
    B, N, H_kv, d, page, start, n_new = shape
    pool, dpool, k, v, n = run_append(18, *shape, rot=rot, layout=layout)
    pos = torch.tensor(start)[:, None] + torch.arange(N)
    turned = ref.rope(k, pos, ref.angles(rot), layout)
    gs = dpool[2].cpu().to(F64)
    gc = as64(dpool[0])
    wc, ws = as64(pool[0]), pool[2].to(F64).clone()
    ref.append(wc, ws, pool[4], turned, start, n, page)
    assert (gs / ws).log2().abs().max() <= 1.0  # another power of two only if the largest value is next to the border
    for b in range(B):
        for i in range(n[b]):
            t = start[b] + i
            p, slot = int(pool[4][b, t // page]), t % page
            got = gc[p, :, slot] * gs[p][:, None]
            want = turned[b, :, i]
            err = 2.0 ** -21 * (2 * k[b, :, i].to(F64).abs().amax(-1, keepdim=True))
            bound = torch.maximum(want.abs() * 2.0 ** -4, gs[p][:, None] * 2.0 ** -10) + err * (1 + 2.0 ** -4)
            assert ((got - want).abs() <= bound).all()
            assert (want.abs().amax(-1) <= 448 * gs[p] * (1 + 2.0 ** -20)).all()
    # values are exact, and so is what was there
    wc, ws = as64(pool[1]), pool[3].to(F64).clone()
    ref.append(wc, ws, pool[4], v.to(F64), start, n, page)
    assert torch.equal(as64(dpool[1]), wc) and torch.equal(dpool[3].cpu().to(F64), ws)


def test_append_infinities_nan_zeros_and_extremes():
    def special(x):
        x[0, 3, :, 0, 5] = math.inf
        x[0, 4, :, 0, 6] = -math.inf
        x[0, 5, :, 1, 7] = math.nan
        x[1] = 0.0
        x[2] = 3.0e38
        x[3] = 1.0e-38
        x[3, 0] = 2.0 ** -95
    shape = (4, 40, 2, 64, 16, [0, 3, 16, 8], None)
    pool, dpool, k, v, n = run_append(19, *shape, x_of=special)
    B, N, H_kv, d, page, start, n_new = shape
    for codes, scales, x, gc, gs in ((pool[0], pool[2], k, dpool[0], dpool[2]), (pool[1], pool[3], v, dpool[1], dpool[3])):
        wc, ws = as64(codes), scales.to(F64).clone()
        ref.append(wc, ws, pool[4], x.to(F64), start, n, page)
        assert torch.equal(gs.cpu().to(F64), ws)
        got = as64(gc)
        assert torch.equal(torch.isnan(got), torch.isnan(wc)) and torch.equal(got.nan_to_num(), wc.nan_to_num())
        assert torch.isnan(got).sum() == 3 and ws.min() == 2.0 ** -100


@pytest.mark.parametrize("shape", [(1, 200, 1, 256, 128, [5], None), (2, 1, 2, 128, 64, [3, 64], None), (1, 70, 2, 128, 64, [0], None)])
@pytest.mark.parametrize("offset", [0, 1])
def test_append_infinities_in_every_kernel(shape, offset):
    """Pages read twice, few tokens, and heads without infinities next to heads with them."""
    def special(x):
        x[0, 0, 0, 0, 7] = math.inf
        x[0, -1, 1, -1, 9] = -math.inf
        x[0, -1, 0, 0, 11] = math.nan
    B, N, H_kv, d, page, start, n_new = shape
    pool, dpool, k, v, n = run_append(47, *shape, x_of=special, offset=offset)
    for codes, scales, x, gc, gs in ((pool[0], pool[2], k, dpool[0], dpool[2]), (pool[1], pool[3], v, dpool[1], dpool[3])):
        wc, ws = as64(codes), scales.to(F64).clone()
        ref.append(wc, ws, pool[4], x.to(F64), start, n, page)
        assert torch.equal(gs.cpu().to(F64), ws)
        got = as64(gc)
        assert torch.equal(torch.isnan(got), torch.isnan(wc)) and torch.equal(got.nan_to_num(), wc.nan_to_num())


def test_append_behind_a_scale_of_zero():
    """A page whose scale is 0 holds zeros whatever its codes are, also when it gets a scale."""
    H_kv, d, page = 1, 64, 16
    for N in (1, 12):  # the kernel for few tokens and the other
        kc, vc = (torch.full((1, H_kv, page, d), 0x38, dtype=torch.uint8, device=dev()) for _ in range(2))
        ks, vs = (torch.zeros(1, H_kv, device=dev()) for _ in range(2))
        x = torch.ones(1, H_kv, N, d, dtype=BF16, device=dev())
        c = fa.PagedCache(kc, vc, ks, vs, ints([[0]]))
        fa.cache_append(c, x, x, ints([3]))
        k, v = fa.cache_gather(c, ints([3 + N]), 3 + N)
        for t in (k, v):
            assert (t[:, :, :3] == 0).all() and (t[:, :, 3:] == 1).all()


def test_append_token_by_token_matches_a_prompt_scale():
    """Tokens one by one: the page's scale ends as the prompt's, the codes within the roundings on the way."""
    g = torch.Generator().manual_seed(20)
    B, N, H_kv, d, page = 2, 70, 2, 64, 32
    x = torch.randn(B, H_kv, N, d, generator=g) * torch.exp(torch.linspace(-2, 2, N))[:, None]
    x = x.to(BF16).to(dev())
    empty = (torch.zeros(8, H_kv, page, d, dtype=torch.uint8), torch.zeros(8, H_kv, page, d, dtype=torch.uint8),
             torch.full((8, H_kv), math.nan), torch.full((8, H_kv), math.nan), torch.arange(8, dtype=torch.int32).view(2, 4))
    one, many = to_gpu(empty), to_gpu(empty)
    fa.cache_append(fa.PagedCache(*many), x, x, ints([0, 0]))
    c = fa.PagedCache(*one)
    for t in range(N):
        fa.cache_append(c, x[:, :, t:t + 1], x[:, :, t:t + 1], ints([t, t]))
    used = [0, 1, 2, 4, 5, 6]
    assert torch.equal(one[2][used], many[2][used]) and torch.equal(one[3][used], many[3][used])
    a, b = (t[0].view(torch.float8_e4m3fn)[used].float() * t[2][used][..., None, None] for t in (one, many))
    # each growth of the scale may round a subnormal code by half its step (2^-10 of the final scale or less,
    # halving with each: 2^-9 in all); both start within half a step of the value
    bound = torch.maximum(b.abs() * 2.0 ** -3, 2.0 ** -8 * many[2][used][..., None, None])
    assert ((a - b).abs() <= bound).all()


def test_append_bad_pages_are_not_written():
    B, N, H_kv, d, page = 4, 40, 1, 64, 16
    g = torch.Generator().manual_seed(21)
    x = torch.randn(B, H_kv, N, d, generator=g).to(BF16).to(dev())
    table = torch.arange(12, dtype=torch.int32).view(4, 3)
    table[0, 1], table[1, 2] = -1, 12
    start = [0, 0, -5, 30]  # the third before the cache, the last past the table
    kc, vc = (Guarded((12, H_kv, page, d), torch.uint8, dev(), fill=1) for _ in range(2))
    ks, vs = (Guarded((12, H_kv), F32, dev(), fill=1.0) for _ in range(2))
    status = ints([0])
    fa.cache_append(fa.PagedCache(kc.t, vc.t, ks.t, vs.t, table.to(dev())), x, x, ints(start), dev_status=status)
    assert fa.read_device_status(status) == fb.FA_ERR_BAD_PAGE
    for t in (kc, vc, ks, vs):
        t.check("pool")
    untouched = [1, 5, 6, 7, 8, 9]
    assert (kc.t[untouched] == 1).all() and (vs.t[untouched] == 1.0).all()
    for p in (0, 2, 3, 4):
        assert (kc.t[p] != 1).any()
    # the last sequence's tokens begin in slot 14 of its second page
    assert (kc.t[10, :, :14] == 1).all() and (kc.t[10, :, 14:] != 1).any() and (kc.t[11] != 1).any()


# ---------------------------------------------------------------- gather
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("lens,N_k", [([0, 1, 300], 300), ([5, 17, 129], 131), ([700], 64), ([3], 1)])
def test_gather(d, page, lens, N_k):
    pool = ref.pool(23, lens, 3, page, d)
    c = cache_of(pool)
    out = [Guarded((len(lens), 3, N_k, d), BF16, dev(), fill=float("nan")) for _ in range(2)]
    status = ints([0])
    fa.cache_gather(c, ints(lens), N_k, out=(out[0].t, out[1].t), dev_status=status)
    assert fa.read_device_status(status) == fb.FA_OK
    for o, codes, scales in ((out[0], pool[0], pool[2]), (out[1], pool[1], pool[3])):
        o.check("gather")
        for b, n in enumerate(lens):
            m = min(n, N_k)
            assert torch.equal(o.t[b, :, :m].cpu().to(F64), ref.dense(codes.float(), scales, pool[4], b, m, page))
            assert (o.t[b, :, m:] == 0).all()


def test_gather_bad_pages_and_long_lengths():
    pool = ref.pool(24, [64, 64], 1, 16, 64)
    pool[4][0, 1], pool[4][1, 3] = -7, 1 << 20
    status = ints([0])
    k, v = fa.cache_gather(cache_of(pool), ints([1000, 64]), 80, dev_status=status)  # the table ends at 64
    assert fa.read_device_status(status) == fb.FA_ERR_BAD_PAGE
    assert (k[0, :, 16:32] == 0).all() and (k[1, :, 48:64] == 0).all() and (k[:, :, 64:] == 0).all()
    assert torch.equal(v[0, :, :16].cpu().to(F64), ref.dense(pool[1].float(), pool[3], pool[4], 0, 16, 16))


# ---------------------------------------------------------------- attention over the cache
def check_attention(o, lse, q, pool, lens, causal, scale, page, live=None):
    """live: for each sequence the tokens that count (default all)."""
    k, v, top_v = [], [], []
    for b, n in enumerate(lens):
        kk = ref.dense(pool[0].float(), pool[2], pool[4].clamp(min=0), b, n, page)
        vv = ref.dense(pool[1].float(), pool[3], pool[4].clamp(min=0), b, n, page)
        k.append(kk)
        v.append(vv)
        top_v.append(vv.nan_to_num().abs().amax() if n else torch.zeros(()))
    want, wl, oabs, mag = ref.attend(q, k, v, lens, causal, scale)
    got, gl = o.cpu().to(F64), lse.cpu().to(F64)
    empty = torch.isneginf(wl)
    assert torch.equal(torch.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    e_x = mag * 2.0 ** -21
    far = torch.stack([t.to(F64) for t in top_v]) * torch.tensor(lens, dtype=F64) * 2.0 ** -31
    # top_v bounds max_j (p_j vs_j) 448 up to the 448 / (page's largest code), at most 2^7 for these codes
    rel = (2 * e_x + 2.0 ** -11 + 2.0 ** -18)[..., None]
    bound = rel * (oabs + want.abs()) + far[:, None, None, None] * 128
    bound = bound + (bound + want.abs()) * (2.0 ** -8 if o.dtype == BF16 else 2.0 ** -24)
    err = (got - want).abs()
    assert (err <= bound).all(), (float((err - bound).nan_to_num(9e9).max()), float(err.nan_to_num(9e9).max()))
    lerr = (gl - wl).abs()[~empty]
    assert (lerr <= (e_x + 2.0 ** -18 + 2.0 ** -23 * wl.abs())[~empty]).all(), float(lerr.max())


def run_attention(q, pool, lens, causal, scale, out_dtype=F32, status_want=fb.FA_OK, cache=None, stream=None):
    c = cache or cache_of(pool)
    B, H, N, d = q.shape
    og, lg = Guarded(q.shape, out_dtype, dev(), fill=float("nan")), Guarded(q.shape[:3], F32, dev(), fill=float("nan"))
    ws = Guarded((max(fa.cache_attention_workspace_bytes(c, H, N), 16) // 4,), F32, dev(), fill=float("nan"))
    status = ints([0])
    fa.cache_attention(c, q.to(dev()), ints(lens), causal, scale, out=(og.t, lg.t), workspace=ws.t, dev_status=status,
                       stream=stream)
    assert fa.read_device_status(status) == status_want
    og.check("o")
    lg.check("lse")
    ws.check("workspace")
    return og.t, lg.t


ATTN_SHAPES = [  # H, H_kv, N, d, page, lens
    (1, 1, 1, 64, 16, [1]), (8, 2, 1, 128, 64, [500]), (8, 8, 1, 128, 16, [0, 1, 15, 16, 17, 200]),
    (6, 2, 5, 64, 16, [3, 5, 100, 0]), (16, 2, 1, 256, 32, [33, 700]), (32, 4, 2, 128, 128, [1000, 5, 129]),
    (12, 1, 7, 64, 64, [64, 300]), (8, 1, 7, 256, 16, [90]), (24, 3, 7, 128, 32, [31, 260, 2]), (4, 4, 130, 64, 64, [130, 200, 60]),
    (3, 1, 1, 128, 128, [9000]), (5, 5, 3, 256, 64, [1, 2, 3, 4, 63, 64, 65, 66]),
    (17, 1, 1, 128, 64, [300, 9000]), (8, 1, 4, 64, 32, [64, 3, 7000]), (11, 1, 3, 128, 16, [40, 0, 2]), (4, 1, 9, 256, 128, [130, 4000]),
    (8, 1, 8, 128, 128, [5000, 20]), (10, 2, 4, 64, 16, [100] * 40),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ATTN_SHAPES)
def test_attention(shape, out_dtype, causal):
    H, H_kv, N, d, page, lens = shape
    g = torch.Generator().manual_seed(29)
    pool = ref.pool(31, lens, H_kv, page, d)
    q = torch.randn(len(lens), H, N, d, generator=g).to(BF16)
    o, lse = run_attention(q, pool, lens, causal, d ** -0.5, out_dtype)
    check_attention(o, lse, q, pool, lens, causal, d ** -0.5, page)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,N", [(4, 1), (8, 1), (6, 3)])
@pytest.mark.parametrize("cap", [1, 100, 1000, 3000, 7000])
def test_attention_clusters(d, H, N, cap):
    """One to eight CTAs for a pair, by what the table can hold; most of it empty, or full."""
    lens = [cap, 1, 0, cap // 2]
    g = torch.Generator().manual_seed(d + cap)
    pool = ref.pool(cap, lens, 1, 16, d)
    q = torch.randn(4, H, N, d, generator=g).to(BF16)
    o, lse = run_attention(q, pool, lens, True, d ** -0.5)
    check_attention(o, lse, q, pool, lens, True, d ** -0.5, 16)


@pytest.mark.parametrize("lens", [[70_001], [40_000, 3, 25_000], [129] * 67])
def test_attention_many_parts(lens):
    g = torch.Generator().manual_seed(30)
    pool = ref.pool(32, lens, 1, 128, 64)
    q = torch.randn(len(lens), 2, 1, 64, generator=g).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.125)
    check_attention(o, lse, q, pool, lens, True, 0.125, 128)


def test_attention_scores_that_grow_and_fall():
    """Rows whose maximum comes first, last, and in steps: the references are raised tile by tile."""
    H, d, page, n = 4, 64, 16, 512
    pool = ref.pool(33, [n], 1, page, d)
    ramp = torch.linspace(-40, 40, n // page)
    for sign in (1.0, -1.0):
        order = pool[4][0].long()
        pool[0][order] = ((ramp * sign)[:, None, None, None].expand(-1, 1, page, d) + torch.randn(n // page, 1, page, d,
                          generator=torch.Generator().manual_seed(1))).to(ref.E4M3)
        pool[2].fill_(0.25)
        q = torch.rand(1, H, 1, d, generator=torch.Generator().manual_seed(2)).add(0.5).to(BF16)
        o, lse = run_attention(q, pool, [n], True, 0.125)
        check_attention(o, lse, q, pool, [n], True, 0.125, page)


def test_attention_scales_far_apart_and_no_powers_of_two():
    H, H_kv, d, page, lens = 4, 2, 64, 16, [300, 77]
    g = torch.Generator().manual_seed(34)
    pool = ref.pool(34, lens, H_kv, page, d, spread=(-30, 20))
    pool[2].copy_(0.01 + 0.02 * torch.rand(pool[2].shape, generator=g))
    q = torch.randn(2, H, 1, d, generator=g).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.125)
    check_attention(o, lse, q, pool, lens, True, 0.125, page)
    # pages without any weight (scale 0) count in the sum alone
    pool[3].copy_(0.3 * torch.rand(pool[3].shape, generator=g))
    pool[3][pool[4][0, :5].long()] = 0.0
    o, lse = run_attention(q, pool, lens, True, 0.125)
    check_attention(o, lse, q, pool, lens, True, 0.125, page)


@pytest.mark.parametrize("mag", [2.0 ** 100, 2.0 ** -100, 2.0 ** -126])
def test_attention_queries_of_any_size(mag):
    pool = ref.pool(35, [200], 2, 32, 128)
    scale = 2.0 ** 20 if mag < 1 else 1.0
    fix = min(max(0.05 / mag / scale, 2.0 ** -99), 2.0 ** 100)
    pool[2].fill_(fix)
    q = (torch.randn(1, 4, 1, 128, generator=torch.Generator().manual_seed(3)).double() * mag).to(BF16)
    o, lse = run_attention(q, pool, [200], True, scale)
    check_attention(o, lse, q, pool, [200], True, scale, 32)


def test_attention_nan_behind_the_end_and_among_later_tokens():
    """A NaN code, key or value, that a row does not see does not reach it; one that it sees does."""
    H, H_kv, N, d, page, lens = 4, 2, 5, 128, 16, [37, 64, 3]
    pool = ref.pool(36, lens, H_kv, page, d)
    clean = tuple(t.clone() for t in pool)
    nan = 0x7f
    for c in pool[:2]:
        raw = c.view(torch.uint8)
        for b, n in enumerate(lens):
            if n % page:
                raw[int(pool[4][b, n // page]), :, n % page:] = nan
    q = torch.randn(3, H, N, d, generator=torch.Generator().manual_seed(4)).to(BF16)
    o, lse = run_attention(q, pool, lens, True, 0.1)
    check_attention(o, lse, q, clean, lens, True, 0.1, page)
    # the token of query 3 of each sequence: queries 0 to 2 do not see it
    for which in (0, 1):
        dirty = tuple(t.clone() for t in pool)
        for b, n in enumerate(lens):
            t = n - N + 3
            if t >= 0:
                dirty[which].view(torch.uint8)[int(pool[4][b, t // page]), :, t % page, 9] = nan
        o2, lse2 = run_attention(q, dirty, lens, True, 0.1)
        assert torch.allclose(o2[:, :, :3], o[:, :, :3], rtol=1e-5, atol=1e-6) and torch.equal(lse2[:, :, :3], lse[:, :, :3])
        for b, n in enumerate(lens):
            if n - N + 3 >= 0:
                if which == 0:
                    assert torch.isnan(o2[b, :, 3:]).all() and torch.isnan(lse2[b, :, 3:]).all()
                else:
                    assert torch.isnan(o2[b, :, 3:, 9]).all() and torch.equal(lse2[b], lse[b])
                    rest = [i for i in range(d) if i != 9]
                    assert torch.isfinite(o2[b][..., rest]).all()


def test_attention_special_queries():
    pool = ref.pool(37, [100], 1, 16, 64)
    q = torch.randn(1, 3, 1, 64, generator=torch.Generator().manual_seed(5)).to(BF16)
    q[0, 1, 0, 7] = math.nan
    q[0, 2, 0, 8] = math.inf
    o, lse = run_attention(q, pool, [100], True, 0.125)
    check_attention(o[:, :1], lse[:, :1], q[:, :1], pool, [100], True, 0.125, 16)
    assert torch.isnan(o[0, 1:]).all() and torch.isnan(lse[0, 1]).all()
    q[0, 1:] = 0.0
    o, lse = run_attention(q, pool, [100], True, 0.125)
    check_attention(o, lse, q, pool, [100], True, 0.125, 16)


def test_attention_bad_pages_are_left_out():
    lens, page = [160, 100], 16
    pool = ref.pool(38, lens, 2, page, 64)
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(6)).to(BF16)
    bad = tuple(t.clone() for t in pool)
    bad[4][0, 3], bad[4][0, 9], bad[4][1] = -1, 1 << 28, -5
    o, lse = run_attention(q, bad, lens, False, 0.125, status_want=fb.FA_ERR_BAD_PAGE)
    left = (pool[0], pool[1], pool[2], pool[3], torch.cat([pool[4][:1, :3], pool[4][:1, 4:9]], 1))
    check_attention(o[:1], lse[:1], q[:1], left, [128], False, 0.125, page)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("drop", [1, 5])
def test_attention_wait_that_runs_out(d, drop):
    """A tile that is never loaded ends the wait for it, with the status and without a hang; the next
    call is sound."""
    lens = [2000]
    pool = ref.pool(46, lens, 1, 16, d)
    c = cache_of(pool)
    q = torch.randn(1, 4, 1, d, generator=torch.Generator().manual_seed(15)).to(BF16)
    status = ints([0])
    # 125 tiles: drop = 5 is past what one of few workers has, so the table is made long for one head
    long = fa.PagedCache(c.k, c.v, c.k_scale, c.v_scale, c.table.repeat(1, 200).contiguous())
    n = ints([2000 * 200])
    fa.cache_attention(long, q.to(dev()), n, True, 0.1, dev_status=status, timeout_ms=20, test_drop_load=drop)
    assert fa.read_device_status(status) == fb.FA_ERR_DEVICE_TIMEOUT
    if drop == 1:  # and with clusters
        status.zero_()
        o, _ = fa.cache_attention(c, q.to(dev()), ints(lens), True, 0.1, dev_status=status, timeout_ms=20, test_drop_load=drop)
        assert fa.read_device_status(status) == fb.FA_ERR_DEVICE_TIMEOUT
        assert torch.isnan(o).all()
    o, lse = run_attention(q, pool, lens, True, 0.1, cache=c)
    check_attention(o, lse, q, pool, lens, True, 0.1, 16)


def test_attention_without_any_page():
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(16)).to(BF16)
    none = torch.zeros(0, 2, 16, 64, dtype=torch.uint8, device=dev()), torch.zeros(0, 2, device=dev())
    for table in (torch.zeros(2, 5), torch.full((2, 3000), -1.0)):
        c = fa.PagedCache(none[0], none[0], none[1], none[1], table.to(torch.int32).to(dev()))
        o, lse = run_attention(q, None, [70, 0], True, 0.1, cache=c, status_want=fb.FA_ERR_BAD_PAGE)
        assert (o == 0).all() and torch.isneginf(lse).all()
        status = ints([0])
        k, v = fa.cache_gather(c, ints([70, 0]), 70, dev_status=status)
        assert fa.read_device_status(status) == fb.FA_ERR_BAD_PAGE and (k == 0).all() and (v == 0).all()
        status.zero_()
        x = torch.zeros(2, 2, 3, 64, dtype=BF16, device=dev())
        fa.cache_append(c, x, x, ints([0, 0]), dev_status=status)
        assert fa.read_device_status(status) == fb.FA_ERR_BAD_PAGE
    # a table without columns: sequences without tokens, for few pairs and for many
    for B in (2, 200):
        kv = torch.zeros(1, 2, 16, 64, dtype=torch.uint8, device=dev())
        one = torch.ones(1, 2, device=dev())
        c = fa.PagedCache(kv, kv, one, one, torch.zeros(B, 0, dtype=torch.int32, device=dev()))
        o, lse = run_attention(q[:1].expand(B, 4, 1, 64).contiguous(), None, [9] * B, True, 0.1, cache=c)
        assert (o == 0).all() and torch.isneginf(lse).all()
    # no sequences, no queries
    c = fa.PagedCache(kv, kv, one, one, torch.zeros(0, 3, dtype=torch.int32, device=dev()))
    n = torch.zeros(0, dtype=torch.int32, device=dev())
    o, lse = fa.cache_attention(c, torch.zeros(0, 4, 1, 64, dtype=BF16, device=dev()), n, True, 0.1)
    assert o.shape == (0, 4, 1, 64) and lse.shape == (0, 4, 1)
    assert fa.cache_gather(c, n, 5)[0].shape == (0, 2, 5, 64)
    fa.cache_append(c, torch.zeros(0, 2, 1, 64, dtype=BF16, device=dev()), torch.zeros(0, 2, 1, 64, dtype=BF16, device=dev()), n)


@pytest.mark.parametrize("B", [33, 257])
def test_attention_many_sequences(B):
    """More sequences than a warp has lanes, most of them short or empty."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    lens[B // 2], lens[-1] = 900, 0
    pool = ref.pool(B, lens, 1, 32, 64)
    wide = (*pool[:4], torch.cat([pool[4], torch.full((B, 400), -1, dtype=torch.int32)], 1))
    q = torch.randn(B, 4, 1, 64, generator=g).to(BF16)
    for p in (pool, wide):
        o, lse = run_attention(q, p, lens, True, 0.125)
        check_attention(o, lse, q, p, lens, True, 0.125, 32)


def test_attention_shared_pages_length_past_the_table_and_strided_table():
    page, d = 32, 128
    pool = ref.pool(39, [200], 2, page, d)
    wide = torch.full((3, 16), -1, dtype=torch.int32)
    wide[:, :7] = pool[4][0]
    table = wide.to(dev())[:, :7]
    kc, vc, ks, vs = to_gpu(pool[:4])
    c = fa.PagedCache(kc, vc, ks, vs, table)
    q = torch.randn(3, 4, 2, d, generator=torch.Generator().manual_seed(7)).to(BF16)
    lens = [200, 7 * page, 1]
    o, lse = run_attention(q, None, [200, 1 << 30, 1], True, 0.1, cache=c)
    check_attention(o, lse, q, (*pool[:4], wide[:, :7]), lens, True, 0.1, page)
    o, lse = run_attention(q, None, [-3, 0, -(1 << 31)], True, 0.1, cache=c)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 codes; the pages in use are its last."""
    page, d, H_kv = 128, 256, 8
    n_pages = (1 << 32) // (page * d * H_kv) + 5
    kc, vc = (torch.zeros(n_pages, H_kv, page, d, dtype=torch.uint8, device=dev()) for _ in range(2))
    ks, vs = (torch.ones(n_pages, H_kv, device=dev()) for _ in range(2))
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32)
    c = fa.PagedCache(kc, vc, ks, vs, table.to(dev()))
    g = torch.Generator().manual_seed(8)
    x = torch.randn(2, 1, H_kv, 200, d, generator=g).to(BF16)
    fa.cache_append(c, x[0].to(dev()), x[1].to(dev()), ints([0]))
    small = tuple(torch.zeros(2, *t.shape[1:], dtype=F64) for t in (kc, vc)) + tuple(torch.ones(2, H_kv, dtype=F64) for _ in "kv")
    at = torch.tensor([[0, 1]])
    for i in range(2):
        ref.append(small[i], small[2 + i], at, x[i].to(F64), [0], [200], page)
    last = [n_pages - 1, n_pages - 3]
    assert torch.equal(kc[last].view(ref.E4M3).cpu().to(F64), small[0])
    assert torch.equal(vs[last].cpu().to(F64), small[3])
    pool = (small[0].float().to(ref.E4M3), small[1].float().to(ref.E4M3), small[2].float(), small[3].float(), at)
    q = torch.randn(1, 8, 1, d, generator=g).to(BF16)
    o, lse = run_attention(q, None, [200], True, 0.06, cache=c)
    check_attention(o, lse, q, pool, [200], True, 0.06, page)
    k, v = fa.cache_gather(c, ints([200]), 200)
    assert torch.equal(v[0].cpu().to(F64), ref.dense(pool[1].float(), pool[3], at, 0, 200, page))


# ---------------------------------------------------------------- together, streams, graphs
def test_prompt_then_decoding():
    """A run as it would be used: the prompt's keys turned and appended, its attention over the gathered
    cache, then tokens one by one, each appended and attended."""
    B, H, H_kv, d, page, steps = 3, 8, 2, 128, 16, 6
    prompt = [45, 16, 1]
    N = max(prompt)
    g = torch.Generator().manual_seed(40)
    scale = d ** -0.5
    rot = fa.Rotary(d, scaling="parts", factor=8.0, original_length=4096.0)
    total = [n + steps for n in prompt]
    pool = ref.pool(41, total, H_kv, page, d)
    dpool = to_gpu(pool)
    c = fa.PagedCache(*dpool)
    qkv = torch.randn(B, N, H + 2 * H_kv, d, generator=g).to(BF16).to(dev())
    q, k, v = (x.transpose(1, 2) for x in (qkv[:, :, :H], qkv[:, :, H:H + H_kv], qkv[:, :, H + H_kv:]))
    lens = ints(prompt)
    fa.cache_append(c, k, v, ints([0] * B), n_new=lens, rotary=rot)
    rq = fa.rope(rot, q)
    gk, gv = fa.cache_gather(c, lens, N)
    o, lse = fa.attention(rq, gk, gv, True, scale, k_len=lens)  # rows behind a prompt's end are not used
    w = ref.angles(d, scaling="parts", factor=8.0, original_length=4096.0)

    def host():
        return tuple(t.cpu() for t in dpool)

    for b, n in enumerate(prompt):
        now = host()
        want, wl, _, _ = ref.attend(rq[b:b + 1, :, :n].cpu(), [ref.dense(now[0].float(), now[2], now[4], b, n, page)],
                                    [ref.dense(now[1].float(), now[3], now[4], b, n, page)], [n], True, scale)
        assert (o[b, :, :n].cpu().double() - want[0]).abs().max() <= 1e-2
        assert (lse[b, :, :n].cpu().double() - wl[0]).abs().max() <= 1e-3
    for step in range(steps):
        have = [n + step for n in prompt]
        x = torch.randn(B, 1, H + 2 * H_kv, d, generator=g).to(BF16).to(dev())
        q, k, v = (t.transpose(1, 2) for t in (x[:, :, :H], x[:, :, H:H + H_kv], x[:, :, H + H_kv:]))
        fa.cache_append(c, k, v, ints(have), rotary=rot)
        rq = fa.rope(rot, q, pos=ints([[h] for h in have]))
        o, lse = fa.cache_attention(c, rq, ints([h + 1 for h in have]), True, scale, out_dtype=BF16)
        check_attention(o, lse, rq.cpu(), host(), [h + 1 for h in have], True, scale, page)
        check_rope(rq, q, torch.tensor([[h] for h in have]), dict(scaling="parts", factor=8.0, original_length=4096.0), d)
        # the key that was appended: its code is next to the turned key
        for b, h in enumerate(have):
            got = ref.dense(dpool[0].float().cpu(), dpool[2].cpu(), pool[4], b, h + 1, page)[:, -1]
            want = ref.rope(k[b:b + 1].cpu(), torch.tensor([[h]]), w)[0, :, 0]
            s = dpool[2].cpu()[int(pool[4][b, h // page])].to(F64)[:, None]
            assert ((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) + 1e-5).all()


def test_results_do_not_depend_on_timing_or_stream():
    lens = [3000, 17, 900]
    pool = ref.pool(43, lens, 2, 64, 128)
    c = cache_of(pool)
    q = torch.randn(3, 8, 1, 128, generator=torch.Generator().manual_seed(9)).to(BF16).to(dev())
    n = ints(lens)
    o, lse = fa.cache_attention(c, q, n, True, 0.1)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):  # calls on three streams at once, each with a workspace of its own
        s = side[i % 3]
        got.append(fa.cache_attention(c, q, n, True, 0.1, stream=s if i % 2 else s.cuda_stream))
    for s in side:
        s.synchronize()
    for a, b in got:
        assert torch.equal(a, o) and torch.equal(b, lse)


@pytest.mark.parametrize("room", [1, 1000])  # clusters; split keys and their merge
def test_graph_of_a_decoding_step(room):
    """One captured step, replayed for growing lengths that only the device knows."""
    B, H, H_kv, d, page = 2, 4, 2, 64, 16
    pool = ref.pool(44, [60, 60], H_kv, page, d)
    pool = (*pool[:4], torch.cat([pool[4]] + [torch.full_like(pool[4], -1)] * (room - 1), 1))
    dpool = to_gpu(pool)
    c = fa.PagedCache(*dpool)
    assert (fa.cache_attention_workspace_bytes(c, H, 1) == 0) == (room == 1)
    rot = fa.Rotary(d)
    x = torch.zeros(B, 1, H + 2 * H_kv, d, dtype=BF16, device=dev())
    q, k, v = (t.transpose(1, 2) for t in (x[:, :, :H], x[:, :, H:H + H_kv], x[:, :, H + H_kv:]))
    have = ints([13, 30])

    def step():
        fa.cache_append(c, k, v, have, rotary=rot)
        rq = fa.rope(rot, q, pos=have.view(B, 1))
        have.add_(1)
        return (rq, *fa.cache_attention(c, rq, have, True, 0.125))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    have.copy_(ints([13, 30]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq, o, lse = step()
    g = torch.Generator().manual_seed(10)
    have.copy_(ints([13, 30]))
    for i in range(8):
        x.copy_(torch.randn(x.shape, generator=g).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        lens = [14 + i, 31 + i]
        assert have.tolist() == lens
        check_attention(o, lse, rq.cpu(), tuple(t.cpu() for t in dpool), lens, True, 0.125, page)
    del graph


def test_binding_refusals_on_the_gpu():
    c = cache_of(ref.pool(45, [20], 2, 16, 64))
    long = fa.PagedCache(c.k, c.v, c.k_scale, c.v_scale, c.table.repeat(1, 2000).contiguous())  # needs scratch
    x = torch.zeros(1, 2, 3, 64, dtype=BF16, device=dev())
    n = ints([0])
    r = fa.Rotary(64)
    bad = [
        lambda: fa.cache_append(c, x.float(), x, n), lambda: fa.cache_append(c, x[:, :1], x[:, :1], n),
        lambda: fa.cache_append(c, x, x[:, :, :2], n), lambda: fa.cache_append(c, x, x, n.long()),
        lambda: fa.cache_append(c, x, x, ints([0, 0])), lambda: fa.cache_append(c, x.cpu(), x, n),
        lambda: fa.cache_append(c, x, x, n.cpu()), lambda: fa.cache_append(c, x, x, n, rotary=3),
        lambda: fa.cache_append(c, x.transpose(2, 3).contiguous().transpose(2, 3), x, n),
        lambda: fa.cache_attention(c, x.float(), n, True, 0.1), lambda: fa.cache_attention(c, x[:, :, ::2], n, True, 0.1),
        lambda: fa.cache_attention(c, x[:, :1], n, True, 0.1), lambda: fa.cache_attention(c, x, n, True, 0.1, out_dtype=torch.float16),
        lambda: fa.cache_attention(c, x, n, True, -0.1), lambda: fa.cache_attention(long, x, n, True, 0.1, workspace=n),
        lambda: fa.cache_attention(c, x, n, True, 0.1, out=(x, x)), lambda: fa.cache_gather(c, n, -1),
        lambda: fa.cache_gather(c, n, 4, out=(x, x)), lambda: fa.cache_gather(c, n.float(), 4),
        lambda: fa.rope(r, x, pos=torch.zeros(1, 3, device=dev())), lambda: fa.rope(r, x, pos=ints([0])),
        lambda: fa.rope(r, x, x[:, :, :1]), lambda: fa.rope(r, x.half()), lambda: fa.rope(r, x, out=x[:, :, :2]),
        lambda: fa.rope(r, x, x.float()), lambda: fa.rope(r, x[0]), lambda: fa.rope(fa.Rotary(128), x),
        lambda: fa.rope(r, x, out=x.float(), out_dtype=BF16), lambda: fa.rope(r, x, out=x[:, :1].clone().expand(1, 2, 3, 64)),
        lambda: fa.rope(r, x, pos0=1 << 40), lambda: fa.cache_gather(c, n, 1 << 40), lambda: fa.cache_attention(c, x, n, True, 1e60),
        lambda: fa.cache_attention(c, x, n, True, 0.1, timeout_ms=-1),
        lambda: fa.PagedCache(c.k[:, :, ::2], c.v[:, :, ::2], c.k_scale, c.v_scale, c.table),
        lambda: fa.PagedCache(c.k, c.v[:2], c.k_scale, c.v_scale, c.table),
        lambda: fa.PagedCache(c.k, c.v, c.k_scale.double(), c.v_scale, c.table),
        lambda: fa.PagedCache(c.k, c.v, c.k_scale, c.v_scale, c.table.long()),
        lambda: fa.PagedCache(c.k.float(), c.v, c.k_scale, c.v_scale, c.table),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, fb.FaError)):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()

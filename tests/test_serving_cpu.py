"""Rotary positions and the paged 8-bit cache without a GPU: the table of fa_rotary_init,
the refusals of the C ABI and of the binding, and the definitions that the GPU tests compare with."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest
import torch

import exact_io_aware_52_b200 as fa
from exact_io_aware_52_b200 import _binding as fb
from exact_io_aware_52_b200 import build as fbuild
from tests import serving_ref as ref


@pytest.fixture(scope="module", autouse=True)
def built():
    fbuild.build()


# ---------------------------------------------------------------- the rotation's table
def _pi():
    """Machin's formula."""
    getcontext().prec = 60

    def arctan_inv(n):
        x, k, total, term = Decimal(1) / n, 1, Decimal(0), Decimal(1) / n
        while abs(term) > Decimal(10) ** -58:
            total += term / k if k % 4 == 1 else -(term / k)
            x /= n * n
            term, k = x, k + 2
        return total
    return 4 * (4 * arctan_inv(5) - arctan_inv(239))


@pytest.mark.parametrize("dim,kw", [
    (128, {}), (64, dict(base=500000.0)), (2, {}), (256, dict(scaling="linear", factor=4.0)),
    (96, dict(scaling="base", factor=8.0)), (128, dict(scaling="parts", factor=20.0, original_length=4096.0)),
])
def test_rotary_steps(dim, kw):
    r = fa.Rotary(dim, **kw)
    getcontext().prec = 60
    pi = _pi()
    base = Decimal(kw.get("base", 10000.0))
    factor = Decimal(kw.get("factor", 1.0))
    kind = kw.get("scaling", "none")
    if kind == "base":
        base *= (factor.ln() * dim / (dim - 2)).exp()
    for i in range(dim // 2):
        w = (base.ln() * Decimal(-2 * i) / dim).exp()
        if kind == "linear":
            w /= factor
        if kind == "parts":
            turns = Decimal(kw["original_length"]) * w / (2 * pi)
            keep = min(max((turns - 1) / 31, Decimal(0)), Decimal(1))
            w = keep * w + (1 - keep) * w / factor
        t = w / (2 * pi) * Decimal(2) ** 64
        # long double arithmetic: 64-bit mantissas, a dozen roundings (the power the largest) of at most one turn
        assert abs(Decimal(int(r.struct.step[i])) - t) <= max(Decimal(1), t * Decimal(2) ** -58)


def test_rotary_own_angles():
    a = [0.5, -0.25, 0.0, 7.0]
    r = fa.Rotary(8, angles=a, amplitude=1.5, layout="interleaved")
    for i, x in enumerate(a):
        turn = (x / (2 * math.pi)) % 1.0
        assert abs(r.struct.step[i] / 2.0 ** 64 - turn) <= 2.0 ** -50
    assert r.struct.amplitude == 1.5


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=3), dict(dim=258), dict(base=0.0), dict(base=-1.0), dict(base=math.inf), dict(base=math.nan),
    dict(scaling="linear", factor=0.0), dict(scaling="base", factor=-2.0), dict(scaling="base", factor=2.0, dim=2),
    dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0, original_length=4096.0, low_turns=32.0),
    dict(scaling="parts", factor=2.0, original_length=4096.0, low_turns=-1.0), dict(angles=[math.nan] * 32),
    dict(angles=[1e9] * 32), dict(angles=[1.0] * 31), dict(layout="whole"), dict(scaling="some"), dict(amplitude=0.0),
    dict(amplitude=-1.0), dict(amplitude=math.inf), dict(base=1e-30),
])
def test_rotary_refusals(kw):
    with pytest.raises((ValueError, fb.FaError)):
        fa.Rotary(**{"dim": 64, **kw})


def test_rotary_null():
    r, spec = fb.FaRotary(), fb.FaRotarySpec(dim=64, base=10000.0)
    lib = fb.load()
    assert lib.fa_rotary_init(None, ctypes.byref(spec)) == fb.FA_ERR_INVALID_ARGUMENT
    assert lib.fa_rotary_init(ctypes.byref(r), None) == fb.FA_ERR_INVALID_ARGUMENT
    assert lib.fa_rotary_init(ctypes.byref(r), ctypes.byref(spec)) == fb.FA_OK


# ---------------------------------------------------------------- refusals of the C ABI
def _rotary(dim=64, **kw):
    return ctypes.pointer(fa.Rotary(dim, **kw).struct)


def _rope_status(**kw):
    p = fb.FaRopeParams(B=2, N=8, d=64, x_dtype=0, y_dtype=0, rotary=kw.pop("rotary", _rotary()))
    p.t[0] = fb.FaRopeTensor(x=0x10000, y=0x20000, heads=4)
    p.t[0].x_stride[:] = p.t[0].y_stride[:] = (2048, 512, 64)
    t0 = kw.pop("t0", {})
    for k, v in t0.items():
        if k.endswith("stride"):
            getattr(p.t[0], k)[:] = v
        else:
            setattr(p.t[0], k, v)
    for k, v in kw.items():
        setattr(p, k, v)
    return fb.load().fa_rope(ctypes.byref(p), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), fb.FA_ERR_INVALID_ARGUMENT), (dict(N=-1), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(x_dtype=2), fb.FA_ERR_INVALID_ARGUMENT), (dict(y_dtype=-1), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(inverse=2), fb.FA_ERR_INVALID_ARGUMENT), (dict(d=1), fb.FA_ERR_UNSUPPORTED),
    (dict(d=1025), fb.FA_ERR_UNSUPPORTED), (dict(d=62), fb.FA_ERR_INVALID_ARGUMENT),  # the rotation is wider
    (dict(rotary=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(rotary=ctypes.pointer(fb.FaRotary(dim=64))), fb.FA_ERR_INVALID_ARGUMENT),  # not initialised
    (dict(t0=dict(x=None)), fb.FA_ERR_INVALID_ARGUMENT), (dict(t0=dict(y=None)), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(t0=dict(heads=-1)), fb.FA_ERR_INVALID_ARGUMENT), (dict(t0=dict(heads=70000)), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(B=1 << 20, N=1 << 20), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(t0=dict(x=0x10001)), fb.FA_ERR_MISALIGNED), (dict(pos=0x30002), fb.FA_ERR_MISALIGNED),
    (dict(x_dtype=1, t0=dict(x=0x10002)), fb.FA_ERR_MISALIGNED),
    (dict(t0=dict(y=0x10000, y_stride=(2048, 64, 256))), fb.FA_ERR_INVALID_ARGUMENT),  # in place, other strides
    (dict(y_dtype=1, t0=dict(y=0x10000)), fb.FA_ERR_INVALID_ARGUMENT),               # in place, other type
    (dict(t0=dict(heads=0)), fb.FA_OK), (dict(B=0), fb.FA_OK), (dict(N=0), fb.FA_OK),
])
def test_rope_refusals(kw, expect):
    assert _rope_status(**kw) == expect


def _cache(**kw):
    base = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, table=0x50000, table_stride=8, n_pages=16,
                max_pages=8, B=2, H_kv=2, page=64, d=128)
    base.update(kw)
    return fb.FaCache(**base)


CACHE_REFUSALS = [
    (dict(B=-1), fb.FA_ERR_INVALID_ARGUMENT), (dict(H_kv=-1), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(n_pages=-1), fb.FA_ERR_INVALID_ARGUMENT), (dict(max_pages=-1), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(table_stride=-8), fb.FA_ERR_INVALID_ARGUMENT), (dict(page=48), fb.FA_ERR_UNSUPPORTED),
    (dict(page=8), fb.FA_ERR_UNSUPPORTED), (dict(page=256), fb.FA_ERR_UNSUPPORTED), (dict(d=96), fb.FA_ERR_UNSUPPORTED),
    (dict(d=0), fb.FA_ERR_UNSUPPORTED), (dict(max_pages=1 << 30), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(B=1 << 20, H_kv=1 << 20), fb.FA_ERR_INVALID_ARGUMENT), (dict(n_pages=1 << 30, H_kv=8), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(k=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(v=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(k_scale=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(v_scale=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(table=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(k=0x10008), fb.FA_ERR_MISALIGNED),
    (dict(v=0x20001), fb.FA_ERR_MISALIGNED), (dict(k_scale=0x30002), fb.FA_ERR_MISALIGNED),
    (dict(table=0x50001), fb.FA_ERR_MISALIGNED), (dict(B=0), fb.FA_OK), (dict(H_kv=0), fb.FA_OK),
]


def _append_status(cache=None, **kw):
    base = dict(cache=_cache(**(cache or {})), k=0x60000, v=0x70000, N=4, start=0x80000)
    base.update(kw)
    p = fb.FaCacheAppendParams(**base)
    p.k_stride[:] = p.v_stride[:] = (1024, 512, 128)
    return fb.load().fa_cache_append(ctypes.byref(p), None)


def _gather_status(cache=None, **kw):
    base = dict(cache=_cache(**(cache or {})), k_len=0x80000, k=0x60000, v=0x70000, N_k=100)
    base.update(kw)
    return fb.load().fa_cache_gather(ctypes.byref(fb.FaCacheGatherParams(**base)), None)


def _attn_params(cache=None, **kw):
    base = dict(cache=_cache(**{"max_pages": 512, **(cache or {})}), q=0x60000, o=0x70000, lse=0x80000, k_len=0x90000, H=8, N=1, causal=1,
                scale=0.1, o_dtype=0, workspace=0xa0000, workspace_bytes=1 << 30)
    base.update(kw)
    return fb.FaCacheAttnParams(**base)


def _attn_status(cache=None, **kw):
    return fb.load().fa_cache_attn(ctypes.byref(_attn_params(cache, **kw)), None)


@pytest.mark.parametrize("call", [_append_status, _gather_status, _attn_status])
@pytest.mark.parametrize("cache,expect", CACHE_REFUSALS)
def test_cache_refusals(call, cache, expect):
    assert call(cache) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), fb.FA_ERR_INVALID_ARGUMENT), (dict(N=0), fb.FA_OK), (dict(k=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(v=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(start=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(k=0x60001), fb.FA_ERR_MISALIGNED), (dict(start=0x80002), fb.FA_ERR_MISALIGNED),
    (dict(n_new=0x80002), fb.FA_ERR_MISALIGNED), (dict(dev_status=0x80002), fb.FA_ERR_MISALIGNED),
    (dict(rotary=ctypes.pointer(fb.FaRotary(dim=64))), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(rotary=_rotary(256)), fb.FA_ERR_INVALID_ARGUMENT),  # wider than the head
])
def test_append_refusals(kw, expect):
    assert _append_status(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(N_k=-1), fb.FA_ERR_INVALID_ARGUMENT), (dict(N_k=0), fb.FA_OK), (dict(k=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(v=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(k_len=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(k=0x60008), fb.FA_ERR_MISALIGNED), (dict(v=0x70002), fb.FA_ERR_MISALIGNED),
    (dict(k_len=0x80002), fb.FA_ERR_MISALIGNED),
])
def test_gather_refusals(kw, expect):
    assert _gather_status(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(H=-8), fb.FA_ERR_INVALID_ARGUMENT), (dict(N=-1), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(H=3), fb.FA_ERR_INVALID_ARGUMENT), (dict(causal=2), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(scale=0.0), fb.FA_ERR_INVALID_ARGUMENT), (dict(scale=math.nan), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(scale=math.inf), fb.FA_ERR_INVALID_ARGUMENT), (dict(scale=-1.0), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(o_dtype=2), fb.FA_ERR_INVALID_ARGUMENT), (dict(q=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(o=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(lse=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(k_len=None), fb.FA_ERR_INVALID_ARGUMENT), (dict(workspace=None), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(workspace_bytes=16), fb.FA_ERR_INVALID_ARGUMENT), (dict(q=0x60008), fb.FA_ERR_MISALIGNED),
    (dict(o=0x70004), fb.FA_ERR_MISALIGNED), (dict(lse=0x80002), fb.FA_ERR_MISALIGNED),
    (dict(workspace=0xa0008), fb.FA_ERR_MISALIGNED), (dict(test_drop_load=-1), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(H=1 << 20, N=1 << 20), fb.FA_ERR_INVALID_ARGUMENT),
    (dict(H=0), fb.FA_OK), (dict(N=0), fb.FA_OK),
])
def test_attn_refusals(kw, expect):
    assert _attn_status(**kw) == expect


def test_null_params():
    lib = fb.load()
    for f in (lib.fa_rope, lib.fa_cache_append, lib.fa_cache_gather, lib.fa_cache_attn):
        assert f(None, None) == fb.FA_ERR_INVALID_ARGUMENT
    assert lib.fa_cache_attn_workspace_bytes(None) == 0


def test_attn_workspace_bytes():
    size = lambda cache=None, **kw: fb.load().fa_cache_attn_workspace_bytes(ctypes.byref(_attn_params(cache, **kw)))  # noqa: E731
    # one pair of slots of 4 or 8 rows for each worker, 2560 workers at most
    assert size() == size(dict(B=64, max_pages=128)) == 2560 * 2 * 4 * (128 + 2) * 4
    assert size(H=16) == 2560 * 2 * 8 * (128 + 2) * 4
    # 1000 pairs with 2 tiles each: no more workers than tiles
    assert size(dict(B=500, max_pages=2, page=16)) == 2000 * 2 * 4 * (128 + 2) * 4
    # few sequences that can hold few tokens: none
    assert size(dict(max_pages=8)) == size(dict(B=1, H_kv=1, max_pages=1), H=1) == 0
    assert size(H=0) == size(N=0) == size(H=3) == size(dict(page=5)) == size(dict(B=0)) == 0
    assert fb.status_string(fb.FA_ERR_BAD_PAGE) == "FA_ERR_BAD_PAGE"


# ---------------------------------------------------------------- refusals of the binding
def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.rope(fa.Rotary(64), q)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.ones(4, 2)
    with pytest.raises(ValueError):
        fa.PagedCache(c, c, s, s, torch.zeros(1, 4, dtype=torch.int32))


# ---------------------------------------------------------------- the definitions
def test_page_exponent():
    for e in (-100, -30, -1, 0, 3, 100):
        top = 448.0 * 2.0 ** e
        assert ref.page_exponent(top) == e
        assert ref.page_exponent(top * (1 + 2.0 ** -50)) == e + 1
        assert ref.page_exponent(top / 2 * (1 + 2.0 ** -50)) == e
    assert ref.page_exponent(0.0) == ref.MIN_EXP


def test_codes_rounding_is_e4m3():
    x = torch.cat([torch.linspace(-448, 448, 40001, dtype=torch.float64), torch.linspace(-0.03, 0.03, 4001, dtype=torch.float64)])
    x = x.float().double()  # torch's conversion starts from 32 bits
    assert torch.equal(ref.to_codes(x), x.float().to(ref.E4M3).double())
    assert torch.isnan(ref.to_codes(torch.tensor([math.inf, -math.inf, math.nan], dtype=torch.float64))).all()


def test_rotation_keeps_distance():
    """q . k of turned heads depends on the distance alone, and the inverse undoes the rotation."""
    g = torch.Generator().manual_seed(5)
    q, k = torch.randn(2, 1, 1, 1, 64, generator=g, dtype=torch.float64)
    w = ref.angles(64)
    at = lambda p: torch.tensor([[p]])  # noqa: E731
    for layout in ("half", "interleaved"):
        a = (ref.rope(q, at(17), w, layout) * ref.rope(k, at(5), w, layout)).sum()
        b = (ref.rope(q, at(1012), w, layout) * ref.rope(k, at(1000), w, layout)).sum()
        assert abs(a - b) <= 1e-9
        assert (ref.rope(ref.rope(q, at(99), w, layout), at(99), w, layout, inverse=True) - q).abs().max() <= 1e-12


def test_inverse_is_the_gradient():
    """The inverse rotation against differences of a loss."""
    g = torch.Generator().manual_seed(6)
    x, dy = torch.randn(2, 1, 1, 3, 16, generator=g, dtype=torch.float64)
    pos = torch.tensor([[3, 700, 41]])
    w = ref.angles(8)
    for layout in ("half", "interleaved"):
        grad = ref.rope(dy, pos, w, layout, inverse=True, amplitude=1.25)
        for i in range(x.numel()):
            e = torch.zeros(x.numel(), dtype=torch.float64)
            e[i] = 1e-6
            e = e.view(x.shape)
            num = ((ref.rope(x + e, pos, w, layout, amplitude=1.25) - ref.rope(x - e, pos, w, layout, amplitude=1.25))
                   * dy).sum() / 2e-6
            assert abs(num - grad.flatten()[i]) <= 1e-7

"""The rotation's handle and what a call refuses before anything is launched, without a GPU."""
import copy
import ctypes
import gc
import math
import pickle

import pytest

import exact_io_aware_52_b200 as fa
from exact_io_aware_52_b200 import _binding as fb
from exact_io_aware_52_b200 import build as fbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    fbuild.build()


@pytest.mark.parametrize("amplitude", [1e39, 3.5e38, 1.7e308, 1e-50, 5e-324, 2.0 ** -151])
def test_rotary_refuses_amplitudes_outside_fp32(amplitude):
    """The kernels hold the amplitude in fp32: what becomes an infinity or zero there is refused."""
    with pytest.raises(fb.FaError) as e:
        fa.Rotary(64, amplitude=amplitude)
    assert e.value.status == fb.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("amplitude", [1e38, 3.4028234e38, 2.0 ** -149, 0.7])
def test_rotary_keeps_amplitudes_of_fp32(amplitude):
    got = fa.Rotary(64, amplitude=amplitude).struct.amplitude
    assert math.isfinite(got) and abs(got - amplitude) <= 2.0 ** -24 * amplitude


def test_rotary_amplitude_zero_means_one():
    r, spec = fb.FaRotary(), fb.FaRotarySpec(dim=64, base=10000.0, amplitude=0.0)
    assert fb.load().fa_rotary_init(ctypes.byref(r), ctypes.byref(spec)) == fb.FA_OK and r.amplitude == 1.0


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_copies_of_a_rotation_have_their_own_table(how):
    """A call passes the address of the table: a copy that outlives the rotation it was made from has to pass
    that of a table that lives as long as itself."""
    r = fa.Rotary(64, layout="interleaved", amplitude=1.5, base=500.0)
    want = bytes(r.struct)
    c = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda x: pickle.loads(pickle.dumps(x))}[how](r)
    assert c._address == ctypes.addressof(c.struct) and bytes(c.struct) == want
    assert (c.dim, c.layout) == (64, "interleaved")
    del r
    gc.collect()
    again = [fa.Rotary(64, base=7.0) for _ in range(64)]  # takes the freed table's place, if there is one
    assert ctypes.string_at(c._address, len(want)) == want
    del again


# ---------------------------------------------------------------- refusals of fa_rope
def _rope_status(t0=None, **kw):
    p = fb.FaRopeParams(B=2, N=8, d=64, x_dtype=0, y_dtype=0, rotary=ctypes.pointer(fa.Rotary(64).struct))
    p.t[0] = fb.FaRopeTensor(x=0x10000, y=0x20000, heads=4)
    p.t[0].x_stride[:] = p.t[0].y_stride[:] = (2048, 512, 64)
    for k, v in (t0 or {}).items():
        if k.endswith("stride"):
            getattr(p.t[0], k)[:] = v
        else:
            setattr(p.t[0], k, v)
    for k, v in kw.items():
        setattr(p, k, v)
    return fb.load().fa_rope(ctypes.byref(p), None)


def test_rope_refuses_positions_past_int32():
    """Token n is at pos0 + n, which must not wrap around."""
    last = 2 ** 31 - 1
    assert _rope_status(pos0=last - 6) == fb.FA_ERR_INVALID_ARGUMENT
    assert _rope_status(pos0=last) == fb.FA_ERR_INVALID_ARGUMENT
    assert _rope_status(pos0=last, N=0) == fb.FA_OK  # no token (nothing is launched)


@pytest.mark.parametrize("t0", [
    dict(y_stride=(0, 512, 64)), dict(y_stride=(2048, 0, 64)), dict(y_stride=(2048, 512, 0)),
    dict(y=0x10000, x_stride=(0, 512, 64), y_stride=(0, 512, 64)),  # in place: turned once for each batch element
])
def test_rope_refuses_outputs_whose_entries_share_a_place(t0):
    assert _rope_status(t0) == fb.FA_ERR_INVALID_ARGUMENT


def test_rope_refuses_more_rows_than_its_grid_counts():
    """The grid is counted in 32 bits, with up to 255 rows of a block behind the last one."""
    for B, N in ((1, 2 ** 31 - 1), (1, 2 ** 31 - 255), (2 ** 31 - 255, 1), (2 ** 16, 2 ** 15)):
        assert _rope_status(B=B, N=N) == fb.FA_ERR_INVALID_ARGUMENT

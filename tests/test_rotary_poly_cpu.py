"""The sine and cosine of the rotary kernels, emulated in fp32 on the CPU with the constants of the source: the
figures that its comment gives, which the tests of turned tensors build on."""
import os
import re

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_52_b200", "csrc",
                   "fa_rotary.cuh")
F32, LONG = np.float32, np.longdouble
TWO_PI = LONG("6.283185307179586476925286766559")


def constants():
    """(unit of the angle, sine's from the highest degree, cosine's likewise) as fp32."""
    text = open(SRC).read()
    body = text[text.index("void rotary_cs("):]
    num = r"(-?\d\.\d+(?:e-\d+)?)f"
    unit = re.search(r"\(quarter << 30\)\) \* " + num, body).group(1)
    coeffs = [re.search(rf"float {name} = fmaf\(fmaf\({num}, t, {num}\), t, {num}\)", body).groups() for name in ("sp", "cp")]
    return F32(unit), [F32(x) for x in coeffs[0]], [F32(x) for x in coeffs[1]]


def fma(a, b, c):
    # the product of two fp32 numbers is exact in 64 bits of mantissa, the sum then rounds to those and to fp32
    return (a.astype(LONG) * b.astype(LONG) + c.astype(LONG)).astype(F32)


def test_fp32_steps():
    unit, sc, cc = constants()
    assert abs(LONG(unit) / (TWO_PI * LONG(2) ** -32) - 1) <= LONG(2) ** -24
    rng = np.random.default_rng(0)
    worst = [0.0, 0.0]
    for part in range(4):
        angle = (rng.integers(0, 2 ** 32, 1 << 20) if part else np.linspace(0, 2 ** 32 - 1, 1 << 20).astype(np.int64)).astype(np.uint32)
        quarter = (angle + np.uint32(0x20000000)) >> np.uint32(30)
        x = (angle - (quarter << np.uint32(30))).view(np.int32).astype(F32) * unit
        t = x * x
        full = lambda v: np.full_like(t, v)  # noqa: E731
        sp = fma(fma(full(sc[0]), t, full(sc[1])), t, full(sc[2]))
        cp = fma(fma(full(cc[0]), t, full(cc[1])), t, full(cc[2]))
        sx = fma(x * t, sp, x)
        cx = fma(fma(cp, t, full(-0.5)), t, full(1.0))
        c = np.choose(quarter & 3, [cx, -sx, -cx, sx])
        s = np.choose(quarter & 3, [sx, cx, -sx, -cx])
        theta = angle.astype(LONG) * TWO_PI * LONG(2) ** -32
        for i, (got, want) in enumerate(((c, np.cos(theta)), (s, np.sin(theta)))):
            worst[i] = max(worst[i], float(np.abs(got.astype(LONG) - want).max()))
    assert max(worst) <= 2.0 ** -23.2
    assert max(worst) >= 2.0 ** -23.6  # the figure is not far above what is measured


@pytest.mark.parametrize("which,absolute", [("sine", 2.0 ** -27.3), ("cosine", 2.0 ** -30.8)])
def test_polynomials(which, absolute):
    """Without the fp32 steps: what the rounding of the coefficients leaves of the fits."""
    _, sc, cc = constants()
    x = np.linspace(0, float(TWO_PI / 8), 100_001).astype(LONG)
    t = x * x
    if which == "sine":
        err = x + x * t * (LONG(sc[2]) + t * (LONG(sc[1]) + t * LONG(sc[0]))) - np.sin(x)
        assert np.abs(err[1:] / np.sin(x[1:])).max() <= 2.0 ** -26.8
    else:
        err = 1 - t / 2 + t * t * (LONG(cc[2]) + t * (LONG(cc[1]) + t * LONG(cc[0]))) - np.cos(x)
    assert np.abs(err).max() <= absolute

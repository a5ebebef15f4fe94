"""The plain references themselves, against exact fractions."""
from fractions import Fraction

import numpy as np

from tests import beamref


def nearest32(f: Fraction) -> np.float32:
    mid = np.float32(float(f))
    near = (mid, np.nextafter(mid, np.float32(np.inf)), np.nextafter(mid, np.float32(-np.inf)))
    return min(near, key=lambda v: (abs(Fraction(float(v)) - f), int(v.view(np.uint32)) & 1))


def test_fused32_rounds_the_exact_sum_once():
    rng = np.random.default_rng(0)
    n = 2000
    a = (rng.standard_normal(n) * 1e4).astype(np.float32)
    b = (rng.standard_normal(n) * 1e-4).astype(np.float32)
    c = (rng.standard_normal(n) * 10.0 ** rng.integers(-9, 9, n)).astype(np.float32)
    p = a.astype(np.float64) * b.astype(np.float64)
    c[::3] = -p[::3].astype(np.float32)  # sums that cancel
    # ends of the addend's last place halved by the product: the sum lies next to a tie
    c[1::3] = (np.float32(1) + np.arange(len(c[1::3]), dtype=np.float32) * np.float32(2.0 ** -23))
    a[1::3], b[1::3] = np.float32(2.0 ** -24), np.float32(1) + np.float32(2.0 ** -23) * rng.integers(-1, 2, len(c[1::3])).astype(np.float32)
    got = beamref.fused32(a, b, c)
    want = [nearest32(Fraction(float(x)) * Fraction(float(y)) + Fraction(float(z))) for x, y, z in zip(a, b, c)]
    assert np.array_equal(got, np.array(want))
    assert (got != a * b + c).any()

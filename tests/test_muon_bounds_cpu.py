"""The bound on the singular values that zds_newton_schulz forms on the host
from a call's coefficients. A call without a plan is refused for that only
behind the coefficients, so both answers show here without a device."""

import ctypes
import time

import numpy as np
import pytest

zds = pytest.importorskip("zero_sharded_mixed_tensor_amd.zds", reason="libzds.so not built")


def refused(coef):
    """Whether the coefficients are, as ones that could pass 8."""
    flat = [x for triple in coef for x in triple]
    arr = (ctypes.c_float * len(flat))(*flat)
    assert zds.lib.zds_newton_schulz(None, None, None, zds.ZDS_BF16, arr, len(coef), None, None, 0, None) == zds.ZDS_EINVAL
    assert "past 8" in zds.zds_last_error() or "null plan" in zds.zds_last_error()
    return "past 8" in zds.zds_last_error()


def largest(coef):
    """The largest value of any step by sampling (values of up to 1 to begin
    with, 2^-8 over for rounding in each step), and of b s^2 + c s^4."""
    top, most, mb = 1.0, 0.0, 0.0
    for a, b, c in np.float32(coef).astype(np.float64):
        s = np.linspace(0.0, (1 + 2.0 ** -8) * top, 200_001)
        mb = max(mb, np.abs(b * s ** 2 + c * s ** 4).max())
        top = np.abs(a * s + b * s ** 3 + c * s ** 5).max()
        most = max(most, top)
    return most, mb


def test_bound_against_samples():
    rng = np.random.default_rng(5)
    seen = [0, 0]
    for k in range(600):
        size = 10.0 ** rng.uniform(-1, 1.5, 3)
        coef = (rng.standard_normal((rng.integers(1, 4), 3)) * size)
        coef[:, rng.integers(0, 3)] *= rng.integers(0, 2)      # linear, cubic and odd ones among them
        if k % 3 == 0:
            coef *= 8.0 / max(largest(coef[:1])[0], 1e-9) * rng.uniform(0.98, 1.02)   # next to the border
        most, mb = largest(coef)
        if abs(most / 8 - 1) < 1e-5 or abs(mb / 1e4 - 1) < 1e-5:
            continue
        seen[int(most > 8)] += 1
        assert refused(coef.tolist()) == (most > 8 or mb > 1e4), (coef.tolist(), most, mb)
    assert min(seen) > 100


def test_bound_of_special_coefficients():
    for ok in ((0, 0, 0), (1, 0, 0), (-3.4445, 4.7750, -2.0315), (0, 7, 0), (0, 0, 7), (0, -7, 0), (1e-30, 1e-30, -1e-30)):
        assert not refused([ok]), ok
    inf, nan = float("inf"), float("nan")
    for bad in ((8.1, 0, 0), (0, 8.1, 0), (0, 0, -8.1), (nan, 0, 0), (0, nan, 0), (0, 0, nan), (inf, 0, 0), (0, -inf, 0),
                (0, inf, -inf), (3e38, -3e38, 3e38)):
        assert refused([bad]), bad


def test_bound_takes_no_time():
    """Formed in every call, in front of its first launch (about 5 us each)."""
    arr = (ctypes.c_float * 48)(*([3.4445, -4.7750, 2.0315] * 16))
    least = 1.0
    for _ in range(300):
        t = time.perf_counter()
        zds.lib.zds_newton_schulz(None, None, None, zds.ZDS_BF16, arr, 16, None, None, 0, None)
        least = min(least, time.perf_counter() - t)
    assert least < 40e-6, least


# Steps that start steep and flatten (8.2 times the smallest singular values in the
# first, 1.9 in the last): their values stay below 2, but 2 % more in
# front of every step would take them past 8 in the third.
STEEP = [(8.2052, -22.9018, 16.4607), (4.0664, -2.8612, 0.5184), (3.9096, -2.8234, 0.5250), (3.2856, -2.4153, 0.4853),
         (2.2779, -1.6199, 0.3985), (1.8726, -1.2307, 0.3585), (1.875, -1.25, 0.375)]


def test_steep_coefficients_that_stay_bounded():
    assert largest(STEEP)[0] < 2.1
    for steps in range(1, 8):
        assert not refused(STEEP[:steps])

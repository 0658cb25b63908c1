"""Two scales of a block's sum: their product, or one after the other where that is no
normal number."""
import ctypes
import random
from fractions import Fraction

import numpy as np
import pytest

from tests._host_code import host_library

CODE = r"""
extern "C" float scaled(float p, float a, float b) { return add_scaled(0.0f, p, a, b); }
extern "C" int is_normal(float s) { return normal(s); }
extern "C" float near_scale() { return kNearScale; }
"""
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = host_library(tmp_path_factory.mktemp("scales"), CODE)
    lib.scaled.argtypes, lib.scaled.restype, lib.is_normal.argtypes = [F, F, F], F, [F]
    lib.near_scale.restype = F
    return lib


def _values():
    rng = random.Random(4)
    for _ in range(20000):
        p = float(np.float32(rng.choice([-1, 1]) * rng.uniform(1, 2) * 2.0 ** rng.randrange(-18, 24)))
        a, b = (float(np.float32(rng.choice([-1, 1]) * rng.uniform(1, 2) * 2.0 ** rng.randrange(-148, 127))) for _ in "ab")
        yield p, a, b


def test_every_size_of_scales(lib):
    """Two roundings (2^-24 each) in the normal range, half a smallest step each below it."""
    most = Fraction(float(np.finfo(np.float32).max))
    for p, a, b in _values():
        want = Fraction(p) * Fraction(a) * Fraction(b)
        got = float(lib.scaled(p, a, b))
        if abs(want) > most * (1 - Fraction(1, 2 ** 22)):
            assert got == float("inf") * (1 if want > 0 else -1) or abs(Fraction(got) - want) <= abs(want) / 2 ** 22
        else:
            assert abs(Fraction(got) - want) <= abs(want) * (Fraction(2, 2 ** 24) + Fraction(1, 2 ** 46)) + Fraction(1, 2 ** 149)


def test_normal_numbers(lib):
    info = np.finfo(np.float32)
    most, least = float(info.max), float(info.tiny)
    for v in (least, 1.0, most, float(np.nextafter(info.tiny, np.float32(1)))):
        assert lib.is_normal(v) and lib.is_normal(-v)
    for v in (0.0, 1e-45, float(np.nextafter(info.tiny, np.float32(0))), float("inf"), float("nan")):
        assert not lib.is_normal(v) and not lib.is_normal(-v)


def test_two_near_scales_have_a_normal_product(lib):
    least = lib.near_scale()
    most = float(np.nextafter(np.float32(1 / least), np.float32(0)))
    for a in (least, most, 1.0, 1e-10, -1e10):
        for b in (least, most, 1.0, -1e-10):
            assert lib.is_normal(float(np.float32(a) * np.float32(b)))


def test_zeros_infinities_and_nan(lib):
    inf, nan = float("inf"), float("nan")
    for a, b in ((1e30, 1e30), (1e38, 1e38), (1e-30, 1e-30), (0.0, 1e38), (1e-45, 0.0), (1e38, -1e38)):
        assert lib.scaled(0.0, a, b) == 0
    assert lib.scaled(3.0, inf, 2.0) == inf and lib.scaled(-3.0, 2.0, inf) == -inf and lib.scaled(2.0 ** -18, inf, 1e-45) == inf
    assert np.isnan(lib.scaled(0.0, inf, 2.0)) and np.isnan(lib.scaled(1.0, inf, 0.0)) and np.isnan(lib.scaled(1.0, nan, 0.0))

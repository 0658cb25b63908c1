"""The ranges of keys that the draw divides: every key in one has a part below 512,
whatever the range ends at."""
import ctypes
import random
import struct

import pytest

from tests._host_code import host_library

CODE = r"""
extern "C" int shift(uint32_t lo, uint32_t hi) { return part_shift(lo, hi); }
extern "C" int64_t part(uint32_t key, uint32_t lo, uint32_t hi) {
  return in_range(key, lo, hi) ? (int64_t)part_of(key, hi, part_shift(lo, hi)) : -1;
}
"""
U = ctypes.c_uint32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = host_library(tmp_path_factory.mktemp("ranges"), CODE)
    lib.shift.argtypes, lib.part.argtypes, lib.part.restype = [U, U], [U, U, U], ctypes.c_int64
    return lib


def key(v):  # order_key(v + 0.0f)
    b = struct.unpack("<I", struct.pack("<f", v + 0.0))[0]
    return b ^ 0xffffffff if b >> 31 else b | 0x80000000


LEAST, MOST, MINUS_0 = key(float("-inf")), key(float("inf")), 0x7fffffff


def _ranges():
    rng = random.Random(1)
    ends = [LEAST, MOST, MINUS_0, MINUS_0 - 1, MINUS_0 + 1, key(1e-45), key(-1e-45), key(-1.0), key(1.0)]
    ends += [rng.randrange(LEAST, MOST + 1) for _ in range(40)] + [MINUS_0 + rng.randrange(-5000, 5000) for _ in range(20)]
    return sorted({(min(a, b), max(a, b)) for a in ends for b in ends})


def test_every_key_has_a_part_below_512(lib):
    rng = random.Random(2)
    for lo, hi in _ranges():
        keys = {lo, hi, (lo + hi) // 2, key(0.0), key(-0.0), LEAST, MOST, 0, 0xffffffff, lo - 1, hi + 1 & 0xffffffff}
        keys |= {rng.randrange(lo, hi + 1) for _ in range(20)}
        for k in keys:
            p = lib.part(k, lo, hi)
            assert (0 <= p < 512) if lo <= k <= hi else p == -1, (k, lo, hi)
        s = lib.shift(lo, hi)
        assert (hi - lo) >> s < 512 and (s == 0 or (hi - lo) >> (s - 1) >= 512)


def test_parts_follow_the_order_of_keys(lib):
    rng = random.Random(3)
    for lo, hi in _ranges()[::7]:
        ks = sorted(rng.randrange(lo, hi + 1) for _ in range(50))
        ps = [lib.part(k, lo, hi) for k in ks]
        assert ps == sorted(ps, reverse=True)


def test_zero_is_not_below_zero(lib):
    """A range of the negative values down from the key of -0, whose value +0 is not above."""
    for lo in (MINUS_0 - 3, MINUS_0 - 600, key(-1.0)):
        assert lib.part(key(0.0), lo, MINUS_0) == lib.part(key(-0.0), lo, MINUS_0) == -1
        assert 0 <= lib.part(key(-1e-45), lo, MINUS_0) < 512

"""The quantisation's quotient is the division's, at every pair of a value and a
block's largest value that its rounding can depend on."""
import ctypes

import numpy as np
import pytest

from tests._host_code import host_library

CODE = r"""
// Pairs (x, a) of `bits`-bit significands, x / a in [2^-20, 1], at several exponents of a: how many
// quotients by s = max(a, 2^-96) / 448 from 2^-11 on are not the division's, and the largest otherwise.
extern "C" long pairs(int bits, const int* exponents, int n, float* most) {
  long wrong = 0;
  *most = 0;
  const int one = 1 << (bits - 1);
  for (int e = 0; e < n; ++e)
    for (int am = one; am < 2 * one; ++am) {
      const float a = ldexpf((float)am, exponents[e] - bits + 1);
      const float s = (a < 0x1p-96f ? 0x1p-96f : a) / 448.0f;
      const Quotient by(s);
      for (int down = 0; down <= 20; down += down < 4 ? 1 : 4)
        for (int xm = one; xm < 2 * one; ++xm) {
          float x[2] = {ldexpf((float)xm, exponents[e] - bits + 1 - down), 0.0f};
          if (x[0] > a || x[0] == 0.0f) continue;
          x[1] = -x[0];
          const float want = x[0] / s;
          if (by.tiny) by.divide<true>(x);  // (negated)
          else by.divide<false>(x);
          if (x[1] != -x[0]) ++wrong;
          if (want >= 0x1p-11f) wrong += x[1] != want;
          else if (x[1] > *most) *most = x[1];
        }
    }
  return wrong;
}
extern "C" void one(float scale, float* x) { float v[2] = {*x, *x}; const Quotient by(scale);
  if (by.tiny) by.divide<true>(v); else by.divide<false>(v);
  *x = -v[1]; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = host_library(tmp_path_factory.mktemp("quotient"), CODE)
    lib.pairs.restype = ctypes.c_long
    lib.one.argtypes = [ctypes.c_float, ctypes.POINTER(ctypes.c_float)]
    return lib


@pytest.mark.parametrize("bits,exponents", [(8, [0, 1, 127, 120, 90, -60, -71, -72, -73, -74, -90, -96, -97, -110]),
                                            (11, [0, 15, -13])])
def test_every_pair(lib, bits, exponents):
    e = (ctypes.c_int * len(exponents))(*exponents)
    most = ctypes.c_float()
    assert lib.pairs(bits, e, len(e), ctypes.byref(most)) == 0
    assert most.value < 2.0 ** -11 * (1 + 2.0 ** -22)  # (2^-10 is the first that is not zero's code)


def test_zeros_infinities_and_nan(lib):
    def one(scale, x):
        v = ctypes.c_float(x)
        lib.one(scale, ctypes.byref(v))
        return np.float32(v.value)
    tiny = 2.0 ** -96 / 448
    for s in (tiny, 1.0, 1e30, np.inf):
        for x in (0.0, -0.0):
            assert one(s, x) == 0 and np.signbit(one(s, x)) == np.signbit(x)
    assert one(np.inf, 5.0) == 0 and one(np.inf, -3e38) == 0
    assert np.isnan(one(np.inf, np.inf)) and np.isnan(one(np.nan, 1.0)) and np.isnan(one(np.inf, np.nan))

"""The draw's sums of weights in 32-bit words hold the longest row in one CTA."""
import ctypes

import pytest

from tests._host_code import host_library

CODE = r"""
// n weights w, w + step, w + 2 step, ... (modulo 2^45) added as a CTA adds them; their sum by words.
extern "C" uint64_t added(uint64_t w, uint64_t step, int n) {
  uint32_t sum[kWords] = {};
  for (int i = 0; i < n; ++i, w = (w + step) & ((1ull << kWeightBits) - 1))
    for (int j = 0; j < kWords; ++j) sum[j] += word_of(w, j);
  uint64_t all = 0;
  for (int j = 0; j < kWords; ++j) all += of_word(sum[j], j);
  return all;
}
extern "C" int longest() { return kMaxLogits; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = host_library(tmp_path_factory.mktemp("sums"), CODE)
    lib.added.restype = ctypes.c_uint64
    lib.added.argtypes = [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int]
    return lib


@pytest.mark.parametrize("n", [1, 65536, 131072, 131077, 151936, 196608, 262144, 393216])
@pytest.mark.parametrize("w", [1, 4095, 4096, 32767, 2 ** 30 - 1, 2 ** 44, 2 ** 44 + 2 ** 15 - 1, 2 ** 45 - 2 ** 30, 2 ** 45 - 1])
def test_equal_weights(lib, w, n):
    assert lib.added(w, 0, n) == w * n


@pytest.mark.parametrize("step", [1, 4097, 2 ** 31 + 12345, 2 ** 44 - 7])
def test_unequal_weights(lib, step):
    n, mask = lib.longest(), 2 ** 45 - 1
    assert lib.added(5, step, n) == sum((5 + i * step) & mask for i in range(n))


def test_every_row_is_taken_by_one_cta_or_refused(lib):
    """The rows that moe_sample takes are those whose sums fit."""
    from tests.test_projection_host import SAMPLE, _sample
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as m
    n = lib.longest()
    assert SAMPLE["V"] <= n == 393216 and _sample(m, V=n + 1, stride=n + 1) == 2

"""Borders among the smallest values on either side of zero and among the largest."""
import pytest
import torch

from tests.test_gpu_sample import DEV, F32, BF, _refs, _run, _same, m  # noqa: F401

pytestmark = pytest.mark.gpu


def _asks(V):
    return [(1.0, 0, 0.31073, 0.0), (1.0, 0, 0.77031, 0.0), (1.0, V // 3, 1.0, 0.0), (1.0, V // 2, 0.60017, 0.0),
            (1.0, V - 9, 0.97013, 0.0), (1.0, 40, 0.913, 0.0), (1.0, 0, 0.50317, 0.5), (2.0, V // 5, 1.0, 0.0)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B", [8, 160])
@pytest.mark.parametrize("V", [2000, 40000])
def test_subnormal_values_and_zeros(m, V, B, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(V)
    asks, logits = _asks(V), torch.empty(8, V)
    for i in range(8):
        # whole multiples of the smallest subnormal, of either sign, many of them zeros
        most = (3, 40, 1000, 1 << 22)[i % 4] if dtype is F32 else (3, 40, 90, 120)[i % 4]
        n = torch.randint(-most, most // 3 + 1, (V,), generator=g)
        n[torch.rand(V, generator=g) < 0.3] = 0
        bits = n.abs().to(torch.int32) << (0 if dtype is F32 else 16)
        sign = (n < 0) | ((n == 0) & (torch.rand(V, generator=g) < 0.5))
        bits = torch.where(sign, bits | -2 ** 31, bits)
        logits[i] = bits.view(F32)
    logits = logits.to(dtype)
    us, refs = _refs(logits, asks, g)
    n = B // 8
    _same(_run(m, logits.to(DEV).repeat(n, 1), asks * n, us.repeat(n)), refs * n)


@pytest.mark.parametrize("V", [2000, 40000])
def test_the_largest_values(m, V):  # noqa: F811
    """Temperatures near the largest float: a border's value may not be one."""
    g = torch.Generator().manual_seed(V)
    asks = [(3e38, *a[1:]) for a in _asks(V)]
    logits = torch.empty(8, V).uniform_(-1, 1, generator=g).mul_(torch.finfo(F32).max)
    logits[::2] = torch.where(torch.rand(V, generator=g) < 0.7, torch.finfo(F32).max, logits[::2])
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV), asks, us), refs)

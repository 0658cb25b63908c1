"""Rows whose weights are one value or two, as long as rows get and as many as make a
CTA or two of each: every token of a row adds to one sum."""
import math

import pytest
import torch

from tests._projection_ref import sample_ref
from tests.test_gpu_sample import BF, DEV, F32, FP, _run, _same, m  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(m, rows, asks, B, dtype):  # noqa: F811
    """Every row by every ask, in turn, over B rows; u away from the borders."""
    g = torch.Generator().manual_seed(B)
    logits = torch.stack([rows[i % len(rows)] for i in range(B)])
    us, refs, known = [], [], {}
    for b in range(B):
        key = (b % len(rows), b % len(asks))
        if key not in known:
            ask = tuple(v if i == 1 else float(torch.tensor(v)) for i, v in enumerate(asks[key[1]]))
            for _ in range(9):
                u = float(torch.rand(1, generator=g))
                r = sample_ref(logits[b], *ask, u)
                if r[2] > 2.0 ** -26:
                    break
            assert r[2] > 2.0 ** -26
            known[key] = (u, r)
        us.append(known[key][0])
        refs.append(known[key][1])
    _same(_run(m, logits.to(DEV), [asks[b % len(asks)] for b in range(B)], torch.tensor(us)), refs)


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("B", [3, 130, 259])
@pytest.mark.parametrize("V", [151936, 262144, 393216])
def test_rows_of_one_value(m, V, B, dtype):  # noqa: F811
    rows = [torch.full((V,), v).to(dtype) for v in (0.0, 9.625, -3.3)]
    asks = [(1.0, 0, 0.95, 0.0), (1.0, 0, 0.05, 0.0), (1.0, V // 2, 0.77, 0.0), (0.7, 0, 0.3, 0.0), (1.0, V - 1, 1.0, 0.0)]
    _check(m, rows, asks, B, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B", [130, 259])
@pytest.mark.parametrize("V,first", [(151936, 140000), (262144, 131073), (393216, 300000)])
def test_rows_of_two_values(m, V, first, B, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(V)
    at = torch.randperm(V, generator=g)[:first]
    rows = []
    for high, low in ((0.0, -0.6875), (20.0, 11.5)):
        row = torch.full((V,), low)
        row[at] = high
        rows.append(row.to(dtype))
    asks = [(1.0, 0, 0.2, 0.0), (1.0, 0, 0.93, 0.0), (1.0, 0, 0.9997, 0.0), (1.0, first + 7, 0.61, 0.0), (3.0, first // 2, 1.0, 0.0),
            (1.0, 0, 0.41, 0.5), (1.0, V - 3, 0.99, 0.0)]
    _check(m, rows, asks, B, dtype)


@pytest.mark.parametrize("B", [130, 259])
def test_long_rows_of_few_values(m, B):  # noqa: F811
    """A crowd of one value inside a spread row, in which top-k and top-p end."""
    V = 393216
    g = torch.Generator().manual_seed(B)
    rows = []
    for share in (0.4, 0.9):
        row = torch.randn(V, generator=g) * 2
        row[torch.rand(V, generator=g) < share] = 1.25
        rows.append(row)
    asks = [(1.0, 0, 0.5, 0.0), (1.0, 100000, 0.9, 0.0), (1.0, 150000, 1.0, 0.0), (0.5, 0, 0.7, 1e-3), (2.0, 200000, 0.31, 0.0)]
    _check(m, rows, asks, B, F32)

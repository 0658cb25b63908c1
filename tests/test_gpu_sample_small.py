"""Rows and slices that lie in one 16-byte piece: every top_k of rows of 2 to 17
tokens, and long rows whose last CTA has a few tokens."""
import pytest
import torch

from tests.test_gpu_sample import BF, DEV, F32, FP, _refs, _run, _same, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("off", [0, 1, 2, 3, 5, 7])
def test_every_top_k_of_a_small_row(m, off, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(off)
    for V in range(2, 18):
        asks = [(1.0, k, p, 0.0) for k in range(2, V) for p in (1.0, 0.873) for _ in range(2)] + [(1.0, 0, 0.7, 0.0)]
        wide = torch.full((len(asks), V + 9), 30.0)
        wide[:, off:off + V] = torch.randn(len(asks), V, generator=g)
        wide = wide.to(dtype)
        us, refs = _refs(wide[:, off:off + V], asks, g)
        _same(_run(m, wide.to(DEV)[:, off:off + V], asks, us), refs)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9])
def test_the_last_slice_has_few_tokens(m, n, dtype):  # noqa: F811
    """Eight slices of 3584 tokens but the last: of each of the others as many tokens lead as its
    share of top_k is, then the last's, then the rest."""
    g = torch.Generator().manual_seed(n)
    V = 7 * 3584 + n
    for share in sorted({n, n + 1, 2 * n - 1, 2 * n} - {0}):
        k = 8 * share
        row = torch.rand(V, generator=g) * 0.25
        for c in range(7):
            row[c * 3584 + torch.randperm(3584 // 8, generator=g)[:share] * 8] = 1.0
        row[7 * 3584:] = 0.5
        row = row[None].to(dtype)
        us, refs = _refs(row, [(1.0, k, 1.0, 0.0)], g)
        _same(_run(m, row.to(DEV), [(1.0, k, 1.0, 0.0)], us), refs)

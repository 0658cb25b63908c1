"""Scales whose product is no normal number in some chunks of blocks and not in the
next, in every form of the product, several tiles after one another."""
import pytest
import torch

from tests.test_gpu_linear import DEV, _inputs, _to, m, ws  # noqa: F401
from tests.test_gpu_linear_scales import _check

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("M,N,K", [(3, 700, 5000), (30, 700, 5000), (60, 20480, 1100), (200, 300, 9000), (600, 2999, 2500),
                                   (2100, 2567, 2500), (1100, 4111, 4500)])
def test_some_chunks(m, ws, M, N, K):  # noqa: F811
    g = torch.Generator().manual_seed(M + N)
    x, xs, w, wsc = _inputs(M, N, K, M)
    kb = xs.shape[1]
    hit = torch.rand(M, kb, generator=g) < 0.03
    hit[:, kb // 2:kb // 2 + 2] = False
    for r, b in hit.nonzero().tolist():
        if (r + b) % 3 == 0:  # far below the normal numbers: the block adds nothing that counts
            xs[r, b] = 2.0 ** -130
        elif (r + b) % 3 == 1:  # infinite with a weight block's scale of 2^70: codes of zero
            xs[r, b] = 1e30
            x[r, 128 * b:128 * b + 128] = torch.zeros(min(128, K - 128 * b)).to(x.dtype)
        else:
            xs[r, b] = 0.0
    last = kb - 1  # a weight scale that is large where every row's is small
    wsc[:, last] = 2.0 ** 70
    xs[:, last] = 2.0 ** -75
    a = (x, xs, w, wsc)
    for dtype in (F32, torch.bfloat16):
        out = torch.empty(M, N, device=DEV, dtype=dtype)
        m.moe_linear_e4m3(*_to(a, None), out, ws)
        m.moe_query_status(ws)
        _check(out, a)


@pytest.mark.parametrize("M,N,K", [(2100, 2567, 700), (100, 20480, 2048)])
def test_small_scales_in_large_tiles(m, ws, M, N, K):  # noqa: F811
    g = torch.Generator().manual_seed(M)
    x, xs, w, wsc = _inputs(M, N, K, N)
    xs = xs * torch.exp2(torch.randint(-118, -60, xs.shape, generator=g).float())
    wsc = wsc * torch.exp2(torch.randint(-40, 1, wsc.shape, generator=g).float())
    a = (x, xs, w, wsc)
    out = torch.empty(M, N, device=DEV)
    m.moe_linear_e4m3(*_to(a, None), out, ws)
    m.moe_query_status(ws)
    _check(out, a)

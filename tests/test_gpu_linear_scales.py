"""Scales whose product is no normal fp32 number, beside others whose is: tolerances as
in test_gpu_linear, and half a smallest step for each rounding of a subnormal result."""
import pytest
import torch

from tests._layer_ref import rounded
from tests._projection_ref import linear_ref
from tests.test_gpu_linear import DEV, _inputs, _to, m, ws  # noqa: F401

pytestmark = pytest.mark.gpu
F32 = torch.float32
ROWS = [1, 7, 20, 60, 100, 200, 700]


def _check(out, a):
    ref, mag = linear_ref(*a)
    kb = a[1].shape[1]
    tol = rounded(ref, out.dtype, absolute=mag * ((kb + 8) * 2.0 ** -24 + 2.0 ** -21) + (kb + 9) * 2.0 ** -149)
    err = (out.cpu().double() - ref).abs()
    assert torch.isfinite(out).all() and (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("M", [8, 40, 200])
def test_zero_codes_give_zero_under_two_large_scales(m, ws, M):  # noqa: F811
    x = torch.zeros(M, 32, device=DEV).to(torch.float8_e4m3fn)[:, :20]
    w = torch.ones(130, 32, device=DEV).to(torch.float8_e4m3fn)[:, :20]
    for a, b in ((1e30, 1e30), (3e38, 3e38), (1e-30, 1e-30), (0.0, 3e38)):
        out = torch.full((M, 130), 3.0, device=DEV)
        m.moe_linear_e4m3(x, torch.full((M, 1), a, device=DEV), w, torch.full((2, 1), b, device=DEV), out, ws)
        assert (out == 0).all()


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N,K", [(300, 384), (1000, 4096), (256, 2500)])
def test_small_scales(m, ws, M, N, K):  # noqa: F811
    """Products from far below the smallest subnormal to normal ones, row by row and block by block."""
    g = torch.Generator().manual_seed(M + K)
    x, xs, w, wsc = _inputs(M, N, K, M + N)
    xs = xs * torch.exp2(torch.randint(-118, -60, xs.shape, generator=g).float())
    wsc = wsc * torch.exp2(torch.randint(-40, 1, wsc.shape, generator=g).float())
    xs[::3] = 2.0 ** -140  # a subnormal one
    a = (x, xs, w, wsc)
    for dtype in (F32, torch.bfloat16):
        out = torch.empty(M, N, device=DEV, dtype=dtype)
        m.moe_linear_e4m3(*_to(a, None), out, ws)
        m.moe_query_status(ws)
        _check(out, a)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N,K", [(300, 384), (1000, 4096)])
def test_large_scales_of_small_sums(m, ws, M, N, K):  # noqa: F811
    """Codes of the smallest value, of which few meet: the product of the scales is infinite in
    fp32 and the results are not."""
    g = torch.Generator().manual_seed(M + K)
    x, xs, w, wsc = _inputs(M, N, K, M + N)
    kb = xs.shape[1]
    few = lambda r: ((torch.rand(r, K, generator=g) < 0.02) * 2.0 ** -9).to(torch.float8_e4m3fn)  # noqa: E731
    x.copy_(few(M))
    w.copy_(few(N))
    xs = torch.exp2(torch.randint(60, 64, xs.shape, generator=g).float()) * 1.25
    wsc = torch.exp2(torch.randint(61, 68, wsc.shape, generator=g).float()) * 1.5
    assert kb * 128 * 0.02 * 2.0 ** (64 + 68 - 18 + 1) < 2.0 ** 127
    out = torch.empty(M, N, device=DEV)
    a = (x, xs, w, wsc)
    m.moe_linear_e4m3(*_to(a, None), out, ws)
    _check(out, a)

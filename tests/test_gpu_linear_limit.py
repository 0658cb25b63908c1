"""The least limit of waits that can be set leaves the product's results as they are."""
import pytest
import torch

from tests.test_gpu_linear import DEV, _check, _inputs, _to, m, ws  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 5120, 2048), (40, 2048, 4096), (64, 5120, 8192), (300, 640, 2048), (1500, 2600, 1024)])
def test_the_least_limit(m, ws, M, N, K):  # noqa: F811
    a = _inputs(M, N, K, M)
    d, out = _to(a, None), torch.empty(M, N, device=DEV)
    m.moe_set_wait_timeout_ns(1000)
    try:
        m.moe_linear_e4m3(*d, out, ws)
        m.moe_query_status(ws)
    finally:
        m.moe_set_wait_timeout_ns(2_000_000_000)
    _check(out, a)

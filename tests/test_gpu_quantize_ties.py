"""Codes are those of the fp32 quotient x / s, also where it lies halfway between two
e4m3 values, in blocks of any size of values."""
import pytest
import torch

from tests.test_gpu_quantize import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu


def _codes(x, s, rows):
    T, H = x.shape
    s = s.repeat_interleave(rows, 0)[:T].repeat_interleave(128, 1)[:, :H]
    return (x.float() / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,H,pad", [(700, 2048, 0), (513, 1447, 1), (300, 1000, 4), (2100, 4096, 8), (131, 264, 0)])
def test_codes_are_the_quotients(m, T, H, pad, rows, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H + pad, generator=g).to(dtype)[:, :H]
    x[2::7, ::3] = -0.0
    if dtype is torch.bfloat16:  # tiny and huge blocks
        for i, e in enumerate((-126, -110, -96, -89, -76, -73, -71, 60, 120)):
            x[128 * i:128 * i + 128] = (x[128 * i:128 * i + 128].double() * 2.0 ** e).to(dtype)
    q = torch.empty(T, H + pad, device=DEV, dtype=torch.float8_e4m3fn)[:, :H]
    s = torch.empty(-(-T // rows), -(-H // 128), device=DEV)
    d = torch.empty(T, H + pad, device=DEV, dtype=dtype)[:, :H]
    d.copy_(x)
    m.moe_quantize_e4m3(d, q, s, rows=rows)
    assert torch.equal(q.cpu().contiguous().view(torch.uint8), _codes(x, s.cpu(), rows))

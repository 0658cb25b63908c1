"""Outputs on their own rows' inputs give what they give apart from them; outputs on
other rows' inputs are refused."""
import pytest
import torch

from tests.test_gpu_norm import DEV, EPS, _inputs, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,group", [(1, 2048, 0), (301, 2048, 0), (700, 2048, 128), (3000, 512, 64), (3000, 203, 0),
                                       (700, 1447, 0), (5, 9001, 0), (2, 32768, 0), (41, 16384, 256)])
def test_e4m3_on_the_rows_of_its_input(m, T, H, group):  # noqa: F811
    x, r, w = _inputs(T, H, torch.bfloat16, T + H)
    n = -(-H // group) if group else 1
    want, ws = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(T, n, device=DEV)
    wd = w.to(DEV)
    m.moe_add_rmsnorm(x.to(DEV), wd, want, residual=r.to(DEV), scales=ws, group=group, eps=EPS)
    for on_x in (True, False):
        xd, rd, s = x.to(DEV), r.to(DEV), torch.empty(T, n, device=DEV)
        out = (xd if on_x else rd).view(torch.float8_e4m3fn)[:, :H]  # twice as many bytes from row to row as are used
        m.moe_add_rmsnorm(xd, wd, out, residual=rd, scales=s, group=group, eps=EPS)
        assert torch.equal(out.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, ws)


def test_rows_on_other_rows_are_refused(m):  # noqa: F811
    x, r, w = (t.to(DEV) for t in _inputs(8, 512, torch.bfloat16, 1))
    flat = x.view(torch.float8_e4m3fn).view(-1)[:8 * 512].view(8, 512)
    for kw in (dict(out=flat, scales=torch.empty(8, 1, device=DEV)), dict(out=x, residual=x.flip(0), residual_out=x)):
        before = x.clone()
        with pytest.raises(m.MoeError) as ei:
            m.moe_add_rmsnorm(x, w, **kw)
        assert ei.value.code == 1 and "overlap" in str(ei.value) and torch.equal(x, before)
    wide = torch.empty(9, 512, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(m.MoeError):
        m.moe_add_rmsnorm(wide[:8], w, wide[1:])

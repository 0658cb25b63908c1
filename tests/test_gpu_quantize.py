"""moe_quantize_e4m3 against its 64-bit form.  A scale is one fp32 division
(2^-24 relative); a value is multiplied by the reciprocal of that scale (2^-24
each for scale, reciprocal and product, so under 2^-22) and rounded once to e4m3."""
import math

import pytest
import torch

from tests._projection_ref import quant_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


def _check(q, s, x, rows):
    z, scales = quant_ref(x, rows)
    assert ((s.cpu().double() - scales).abs() <= scales * 2.0 ** -24).all()
    # half a step: 2^-4 relative, 2^-10 among the subnormals
    tol = torch.maximum(z.abs() * (2.0 ** -4 + 2.0 ** -22), torch.tensor(2.0 ** -10)) * (1 + 2.0 ** -22)
    assert ((q.float().cpu().double() - z).abs() <= tol).all()


def _run(m, x, rows, **kw):
    T, H = x.shape
    q = torch.empty(T, H, device=DEV, dtype=torch.float8_e4m3fn)
    s = torch.full((-(-T // rows), -(-H // 128)), math.nan, device=DEV)
    m.moe_quantize_e4m3(x, q, s, rows=rows, **kw)
    return q, s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (3, 7), (2, 2048), (129, 136), (257, 1447), (128, 127), (700, 4096),
                                 (5, 16392), (1300, 264)])
def test_values_and_scales(m, T, H, rows, dtype):
    g = torch.Generator().manual_seed(T + H)
    x = (torch.randn(T, H, generator=g) * (1 + 20 * (torch.rand(H, generator=g) < 0.02))).to(dtype)
    x[0, :128] = 0  # zeros and values below the floor
    if T > 1:
        x[1] *= 2.0 ** -20
    q, s = _run(m, x.to(DEV), rows)
    _check(q, s, x, rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("H,pad,off", [(256, 8, 8), (256, 3, 0), (256, 8, 3), (131, 5, 1), (1000, 24, 16), (9, 0, 1),
                                       (127, 1, 0), (133, 3, 0), (134, 2, 8), (135, 1, 2), (250, 6, 5), (255, 4, 7)])
def test_strides_offsets_and_nothing_beside(m, H, pad, off, rows):
    g = torch.Generator().manual_seed(H + pad)
    T = 133
    wide = torch.randn(T, H + pad + off, generator=g).to(torch.bfloat16)
    out = torch.full((T, H + pad + off), 2.0, device=DEV).to(torch.float8_e4m3fn)
    s = torch.empty(-(-T // rows), -(-H // 128), device=DEV)
    m.moe_quantize_e4m3(wide.to(DEV)[:, off:off + H], out[:, off:off + H], s, rows=rows)
    _check(out[:, off:off + H], s, wide[:, off:off + H], rows)
    f = out.float()
    assert (f[:, :off] == 2).all() and (f[:, off + H:] == 2).all()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("H", [256, 251])
def test_nan_and_infinity_stay_in_their_blocks(m, H, rows):
    g = torch.Generator().manual_seed(H)
    x = torch.randn(256, H, generator=g).to(torch.float16)
    x[3, 5] = math.nan
    x[200, 130] = -math.inf
    q, s = _run(m, x.to(DEV), rows)
    q, s = q.float().cpu(), s.cpu()
    a, b = (3, 200) if rows == 1 else (0, 1)
    bad = torch.zeros_like(s, dtype=torch.bool)
    bad[a, 0] = bad[b, 1] = True
    assert s[a, 0].isnan() and s[b, 1] == math.inf and torch.isfinite(s[~bad]).all()
    ra, rb = (slice(3, 4), slice(200, 201)) if rows == 1 else (slice(0, 128), slice(128, 256))
    assert q[ra, :128].isnan().all()
    block = q[rb, 128:].clone()
    at = (0, 2) if rows == 1 else (72, 2)
    assert block[at].isnan()
    block[at] = 0
    assert (block == 0).all()
    clean = x.clone()
    clean[3, 5] = clean[200, 130] = 0
    q2, s2 = _run(m, clean.to(DEV), rows)
    keep = ~bad.repeat_interleave(rows, 0)[:256].repeat_interleave(128, 1)[:, :H]
    assert torch.equal(q[keep], q2.float().cpu()[keep]) and torch.equal(s[~bad], s2.cpu()[~bad])


def test_no_rows_stream_and_graph(m):
    _run(m, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), 1)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(9, 512, generator=g).to(torch.bfloat16)
    xd = x.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = torch.empty(9, 512, device=DEV, dtype=torch.float8_e4m3fn), torch.empty(9, 4, device=DEV)
    m.moe_quantize_e4m3(xd, q, s, stream=side)
    side.synchronize()
    _check(q, s, x, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_quantize_e4m3(xd, q, s)
    xd.copy_(x.flip(0))
    graph.replay()
    _check(q, s, x.flip(0), 1)

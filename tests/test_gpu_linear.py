"""moe_linear_e4m3 against its 64-bit form.  Products of e4m3 values are exact in
fp32; a block's sum of 128 takes 4 tensor-core steps of 32 terms, each off by at
most a few units of the last place of the sum of magnitudes (2^-21 for the four),
its two scales 2^-23 more, and the sum over the blocks 2^-24 of the magnitudes for
each addition: (blocks + 8) * 2^-24 + 2^-21 in all, then one rounding."""
import math

import pytest
import torch

from tests._layer_ref import rounded
from tests._projection_ref import codes, linear_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


@pytest.fixture(scope="module")
def ws(m):
    return m.alloc_status_workspace(DEV)


def _inputs(M, N, K, seed, pad=None):
    g = torch.Generator().manual_seed(seed)
    kb = -(-K // 128)
    pad = (-K) % 16 if pad is None else pad
    xs = torch.rand(M, kb, generator=g) * 0.01 + 0.002
    wsc = torch.rand(-(-N // 128), kb, generator=g) * 0.01 + 0.002
    return codes(M, K, g, pad), xs, codes(N, K, g, pad), wsc


def _to(a, pads):
    """On the GPU with the same strides."""
    out = []
    for t in a:
        if t.dtype is torch.float8_e4m3fn:
            wide = torch.full((t.shape[0], t.stride(0)), math.nan).to(t.dtype)
            wide[:, :t.shape[1]] = t
            out.append(wide.to(DEV)[:, :t.shape[1]])
        else:
            out.append(t.to(DEV))
    return out


def _check(out, a):
    ref, mag = linear_ref(*a)
    tol = rounded(ref, out.dtype, absolute=mag * ((a[1].shape[1] + 8) * 2.0 ** -24 + 2.0 ** -21))
    err = (out.cpu().double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (2, 129, 130), (7, 5120, 512), (16, 300, 2000), (17, 127, 640), (32, 1000, 4096),
    (33, 257, 48), (64, 520, 1040), (65, 200, 272), (128, 384, 2176), (129, 1, 16), (130, 700, 384), (257, 255, 2100),
    (512, 1447, 256), (777, 256, 2000), (1, 40000, 256), (3, 64, 20000), (300, 64, 5008), (70, 20480, 1024),
    (128, 40001, 512), (90, 300, 70000)])
def test_products(m, ws, M, N, K, dtype):
    a = _inputs(M, N, K, M + N + K)
    out = torch.full((M, N), math.nan, device=DEV, dtype=dtype)
    m.moe_linear_e4m3(*_to(a, None), out, ws)
    m.moe_query_status(ws)
    _check(out, a)


@pytest.mark.parametrize("M", [5, 40, 100, 300])
@pytest.mark.parametrize("stride", [1000, 1001, 1004, 1040])
def test_strided_rows_and_nothing_beside(m, ws, M, stride):
    N, K = 999, 400
    a = _inputs(M, N, K, M, pad=32)
    for dtype in (F32, BF):
        out = torch.full((M + 1, stride), 7.0, device=DEV, dtype=dtype)
        m.moe_linear_e4m3(*_to(a, 32), out[:M, 1:1 + N] if stride > N + 1 else out[:M, :N], ws)
        got = out[:M, 1:1 + N] if stride > N + 1 else out[:M, :N]
        _check(got, a)
        got.fill_(7.0)
        assert (out == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("M,N,K,stride,offset", [
    (600, 2999, 144, 3000, 0), (600, 2999, 300, 3024, 8), (1100, 4111, 272, 4112, 0), (1100, 4111, 130, 4111, 0),
    (1100, 4111, 700, 4128, 16), (2100, 2567, 16, 2570, 1)])
def test_many_rows_of_many_tiles(m, ws, M, N, K, stride, offset, dtype):
    """Several tiles for each pair of SMs, rows that begin on 16 bytes and that do not, nothing beside."""
    a = _inputs(M, N, K, M + K)
    out = torch.full((M + 3, stride), 7.0, device=DEV, dtype=dtype)
    got = out[:M, offset:offset + N]
    m.moe_linear_e4m3(*_to(a, None), got, ws)
    m.moe_query_status(ws)
    _check(got, a)
    got.fill_(7.0)
    assert (out == 7).all()


@pytest.mark.parametrize("M", [3, 20, 64, 100, 200])
def test_nan_and_infinity_reach_only_what_they_are_factors_of(m, ws, M):
    N, K = 300, 384
    a = _inputs(M, N, K, M)
    clean = torch.empty(M, N, device=DEV)
    m.moe_linear_e4m3(*_to(a, None), clean, ws)
    x, xs, w, wsc = (t.clone() for t in a)
    x[1, 200] = math.nan
    xs[2, 1] = math.inf
    w[130, 3] = math.nan
    wsc[2, 2] = math.nan
    out = torch.empty(M, N, device=DEV)
    m.moe_linear_e4m3(*(t.to(DEV) for t in (x, xs, w, wsc)), out, ws)
    hit = torch.zeros(M, N, dtype=torch.bool)
    hit[1:3] = hit[:, 130] = hit[:, 256:] = True
    assert not torch.isfinite(out.cpu()[hit]).any()
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("M", [1, 48, 100, 500])
def test_repeats_give_the_same_bits(m, ws, M):
    a = _to(_inputs(M, 640, 2048, M), None)
    outs = [torch.empty(M, 640, device=DEV) for _ in range(4)]
    for o in outs:
        m.moe_linear_e4m3(*a, o, ws)
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("M", [8, 200])
def test_zero_codes_give_zero_under_any_finite_scale(m, ws, M):
    x = torch.zeros(M, 32, device=DEV).to(torch.float8_e4m3fn)[:, :20]
    w = torch.ones(130, 32, device=DEV).to(torch.float8_e4m3fn)[:, :20]
    out = torch.full((M, 130), 3.0, device=DEV)
    m.moe_linear_e4m3(x, torch.full((M, 1), 1e30, device=DEV), w, torch.ones(2, 1, device=DEV), out, ws)
    assert (out == 0).all()


def test_no_rows_other_stream_and_graph(m, ws):
    a = _inputs(70, 384, 256, 1)
    d = _to(a, None)
    for M, N in ((0, 384), (70, 0)):
        m.moe_linear_e4m3(d[0][:M], d[1][:M], d[2][:N], d[3][:-(-N // 128)], torch.empty(M, N, device=DEV), ws)
    out = torch.empty(70, 384, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_linear_e4m3(*d, out, ws, stream=side)
    side.synchronize()
    _check(out, a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_linear_e4m3(*d, out, ws)
    b = _inputs(70, 384, 256, 2)
    for t, n in zip(d, _to(b, None)):
        t.copy_(n)
    graph.replay()
    _check(out, b)


def test_two_streams_share_a_status_word(m, ws):
    """Two calls at once on one workspace: it holds the status word alone."""
    a, b = _inputs(30, 2000, 2048, 3), _inputs(200, 2000, 2048, 4)
    da, db = _to(a, None), _to(b, None)
    oa, ob = torch.empty(30, 2000, device=DEV), torch.empty(200, 2000, device=DEV)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        m.moe_linear_e4m3(*da, oa, ws, stream=s1)
        m.moe_linear_e4m3(*db, ob, ws, stream=s2)
    torch.cuda.synchronize()
    _check(oa, a)
    _check(ob, b)
    m.moe_query_status(ws)


@pytest.mark.parametrize("M", [4, 150])
def test_the_norms_and_the_quantisations_form(m, ws, M):
    """moe_add_rmsnorm's e4m3 rows with groups of 128 times a quantised weight."""
    g = torch.Generator().manual_seed(M)
    H, N = 1000, 272
    x, w = torch.randn(M, H, generator=g).to(BF), (torch.randn(N, H, generator=g) * 0.02).to(BF)
    q = torch.empty(M, 1008, device=DEV, dtype=torch.float8_e4m3fn)[:, :H]
    s = torch.empty(M, 8, device=DEV)
    m.moe_add_rmsnorm(x.to(DEV), torch.ones(H, dtype=BF, device=DEV), q, scales=s, group=128)
    wq = torch.empty(N, 1008, device=DEV, dtype=torch.float8_e4m3fn)[:, :H]
    wsc = torch.empty(3, 8, device=DEV)
    m.moe_quantize_e4m3(w.to(DEV), wq, wsc, rows=128)
    out = torch.empty(M, N, device=DEV)
    m.moe_linear_e4m3(q, s, wq, wsc, out, ws)
    _check(out, [t.cpu() for t in (q, s, wq, wsc)])
    # against the unquantised product: each factor is off by 2^-4 at most
    y = x.double() * torch.rsqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-6)
    err = (out.cpu().double() - y @ w.double().t()).abs()
    assert (err <= (2 * 2.0 ** -4 + 2.0 ** -7) * (y.abs() @ w.double().abs().t())).all()

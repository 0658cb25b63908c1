"""moe_add_rmsnorm against its 64-bit form.  Errors before the rounding: at most
32 terms in a chain and 10 levels of a tree in the sum of squares, half of that
after the square root, and under 12 further fp32 operations: 2^-19 relative."""
import pytest
import torch

from tests._layer_ref import norm_ref, rounded, scales_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6
REL = 2.0 ** -19


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


def _inputs(T, H, dtype, seed, pad=0, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H + pad, generator=g) * 2).to(dtype)
    r = (torch.randn(T, H + pad, generator=g) * 3).to(dtype) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(dtype)
    return x, r, w


def _check16(out, y, dtype):
    bad = (out.cpu().double() - y).abs() > rounded(y, dtype, REL)
    assert not bad.any(), (out.cpu().double() - y).abs().max()


def _check8(out, scales, y, group):
    s, cols = scales_ref(y, group)
    got = scales.cpu().double()
    assert ((got - s).abs() <= s * 2 * REL).all()
    z = y / cols
    # half a step of 2^-3 relative, or of 2^-9 among the subnormals
    tol = torch.maximum(z.abs() * (2.0 ** -4 + 4 * REL), torch.tensor(2.0 ** -10)) * (1 + 4 * REL)
    assert ((out.cpu().double() - z).abs() <= tol).all()


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 2047), (1, 2048), (33, 4096), (700, 512), (2, 8200), (2, 16384), (1, 32768),
          (3, 32767), (257, 1447), (4, 24)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_sixteen_bits(m, T, H, residual, dtype):
    x, r, w = _inputs(T, H, dtype, T * 7 + H, residual=residual)
    out = torch.empty(T, H, dtype=dtype, device=DEV)
    ro = torch.empty_like(out) if residual else None
    m.moe_add_rmsnorm(x.to(DEV), w.to(DEV), out, residual=r.to(DEV) if residual else None, residual_out=ro, eps=EPS)
    _check16(out, norm_ref(x, w, r, EPS), dtype)
    if residual:
        assert torch.equal(ro.cpu(), (x.float() + r.float()).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,group", [(1, 1, 0), (3, 7, 0), (5, 2047, 0), (1, 2048, 0), (64, 2048, 128), (9, 4096, 64),
                                       (7, 1000, 128), (2, 24, 16), (3, 8200, 256), (2, 32768, 32), (400, 192, 128),
                                       (2, 16384, 0)])
def test_e4m3(m, T, H, group, dtype):
    x, r, w = _inputs(T, H, dtype, T + H)
    x[0] = 0
    r[0] = 0  # a row of zeros: the floor's scale, zeros out
    out = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(T, -(-H // group) if group else 1, device=DEV)
    m.moe_add_rmsnorm(x.to(DEV), w.to(DEV), out, residual=r.to(DEV), scales=scales, group=group, eps=EPS)
    _check8(out.float(), scales, norm_ref(x, w, r, EPS), group)


@pytest.mark.parametrize("H,pad", [(2048, 64), (512, 8), (1000, 24), (1447, 61), (64, 1)])
def test_row_strides_and_offsets(m, H, pad):
    x, r, w = _inputs(19, H, torch.bfloat16, H, pad)
    xd, rd = x.to(DEV), r.to(DEV)
    out = torch.full((19, H + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    ro = torch.full((19, H + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    m.moe_add_rmsnorm(xd[:, pad:], w.to(DEV), out[:, :H], residual=rd[:, :H], residual_out=ro[:, pad:], eps=EPS)
    _check16(out[:, :H], norm_ref(x[:, pad:], w, r[:, :H], EPS), torch.bfloat16)
    assert torch.equal(ro[:, pad:].cpu(), (x[:, pad:].float() + r[:, :H].float()).to(torch.bfloat16))
    assert (out[:, H:] == 7).all() and (ro[:, :pad] == 7).all()


@pytest.mark.parametrize("H", [2048, 1447, 16384])
def test_in_place(m, H):
    x, r, w = _inputs(9, H, torch.float16, H)
    xd, rd = x.to(DEV), r.to(DEV)
    m.moe_add_rmsnorm(xd, w.to(DEV), xd, residual=rd, residual_out=rd, eps=EPS)
    _check16(xd, norm_ref(x, w, r, EPS), torch.float16)
    assert torch.equal(rd.cpu(), (x.float() + r.float()).to(torch.float16))
    xd = x.to(DEV)
    m.moe_add_rmsnorm(xd, w.to(DEV), out := torch.empty_like(xd), residual=rd, residual_out=xd, eps=EPS)
    assert not torch.equal(xd.cpu(), x) and torch.isfinite(out).all()


@pytest.mark.parametrize("H,group", [(2048, 0), (2048, 128), (777, 0)])
def test_nan_and_infinity_stay_in_their_rows(m, H, group):
    x, r, w = _inputs(4, H, torch.bfloat16, H)
    x[1, 5] = float("nan")
    x[2, 3] = float("inf")
    out = torch.empty(4, H, dtype=torch.bfloat16, device=DEV)
    m.moe_add_rmsnorm(x.to(DEV), w.to(DEV), out, residual=r.to(DEV), eps=EPS)
    assert out[1].isnan().all() and out[2, 3].isnan() and (out[2].nan_to_num(0) == 0).all()
    q = torch.empty(4, H, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(4, -(-H // group) if group else 1, device=DEV)
    m.moe_add_rmsnorm(x.to(DEV), w.to(DEV), q, residual=r.to(DEV), scales=s, group=group, eps=EPS)
    assert s[1].isnan().all() and s[2, 0].isnan() and q[1].float().isnan().all()
    for row in (0, 3):
        y = norm_ref(x[row:row + 1], w, r[row:row + 1], EPS)
        _check16(out[row:row + 1], y, torch.bfloat16)
        _check8(q[row:row + 1].float(), s[row:row + 1], y, group)


def test_no_rows_other_stream_and_graph(m):
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    m.moe_add_rmsnorm(e, w, e.clone(), eps=EPS)
    x, _, wt = _inputs(5, 2048, torch.bfloat16, 1)
    xd, wd, out = x.to(DEV), wt.to(DEV), torch.empty(5, 2048, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.moe_add_rmsnorm(xd, wd, out, stream=side)
    side.synchronize()
    _check16(out, norm_ref(x, wt, None, EPS), torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_add_rmsnorm(xd, wd, out)
    x2 = x.flip(0)
    xd.copy_(x2)
    graph.replay()
    _check16(out, norm_ref(x2, wt, None, EPS), torch.bfloat16)


@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 7, 9, 15, 17, 31, 33, 255, 257, 263, 1021, 2049, 4099, 9001])
def test_every_alignment_and_nothing_beside_the_rows(m, H):
    """Rows that start at each place of an 8-byte word, in tensors whose other
    elements must not change."""
    T = 5
    for off in range(4):
        for stride in (H + 4 + off, H + 5 + off):
            x, r, w = _inputs(T, H, torch.bfloat16, H + off)
            xd = torch.full((T, stride), 9.0, dtype=torch.bfloat16, device=DEV)
            rd, od, sd = xd.clone(), xd.clone(), xd.clone()
            wd = torch.zeros(H + off, dtype=torch.bfloat16, device=DEV)
            xd[:, off:off + H], rd[:, 3 - off:3 - off + H], wd[off:] = x.to(DEV), r.to(DEV), w.to(DEV)
            out, ro = od[:, 1:1 + H], sd[:, (off + 2) % 4:(off + 2) % 4 + H]
            m.moe_add_rmsnorm(xd[:, off:off + H], wd[off:], out, residual=rd[:, 3 - off:3 - off + H], residual_out=ro,
                              eps=EPS)
            y = norm_ref(x, w, r, EPS)
            _check16(out, y, torch.bfloat16)
            assert torch.equal(ro.cpu(), (x.float() + r.float()).to(torch.bfloat16))
            rest = torch.ones(T, stride, dtype=torch.bool, device=DEV)
            rest[:, 1:1 + H] = False
            assert (od[rest] == 9).all()
            rest[:] = True
            rest[:, (off + 2) % 4:(off + 2) % 4 + H] = False
            assert (sd[rest] == 9).all()
            for b in (off, off + 4):
                q = torch.full((T, stride + 8), 2.0, device=DEV).to(torch.float8_e4m3fn)
                s = torch.empty(T, 1, device=DEV)
                m.moe_add_rmsnorm(xd[:, off:off + H], wd[off:], q[:, b:b + H], residual=rd[:, 3 - off:3 - off + H],
                                  scales=s, eps=EPS)
                _check8(q[:, b:b + H].float(), s, y, 0)
                qf = q.float()
                assert (qf[:, :b] == 2).all() and (qf[:, b + H:] == 2).all()


@pytest.mark.parametrize("H", [3, 127, 129, 203, 255, 257])
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_narrow_rows(m, H, e4m3):
    T = 5003  # more rows than the SMs hold warps' rows at a time, and no multiple of a CTA's
    x, r, w = _inputs(T, H, torch.float16, H)
    y = norm_ref(x, w, r, EPS)
    out = torch.empty(T, H, dtype=torch.float8_e4m3fn if e4m3 else torch.float16, device=DEV)
    s = torch.empty(T, 1, device=DEV) if e4m3 else None
    m.moe_add_rmsnorm(x.to(DEV), w.to(DEV), out, residual=r.to(DEV), scales=s, eps=EPS)
    if e4m3:
        _check8(out.float(), s, y, 0)
    else:
        _check16(out, y, torch.float16)


@pytest.mark.parametrize("H", [333, 511, 512, 513, 1023, 2047, 6221, 8191])
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_odd_rows(m, H, e4m3):
    """More rows than four per SM, alike and unlike in where they begin."""
    T = 701
    x, r, w = _inputs(T, H, torch.bfloat16, H)
    y = norm_ref(x, w, r, EPS)
    for pad in (0, 1):
        xd = torch.zeros(T, H + pad + 1, dtype=torch.bfloat16, device=DEV)[:, pad:pad + H]
        xd.copy_(x)
        rd = torch.zeros(T, H + pad, dtype=torch.bfloat16, device=DEV)[:, pad:]
        rd.copy_(r)
        out = torch.empty(T, H, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16, device=DEV)
        ro = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        s = torch.empty(T, 1, device=DEV) if e4m3 else None
        m.moe_add_rmsnorm(xd, w.to(DEV), out, residual=rd, residual_out=ro, scales=s, eps=EPS)
        if e4m3:
            _check8(out.float(), s, y, 0)
        else:
            _check16(out, y, torch.bfloat16)
        assert torch.equal(ro.cpu(), (x.float() + r.float()).to(torch.bfloat16))

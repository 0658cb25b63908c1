"""Host-side checks of the quantisation, the 8-bit product and the drawing of
tokens: every refusal of the C entries and of the binding, before anything touches
a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


QUANT = dict(x=1 << 20, out=2 << 20, scales=3 << 20, xs=64, os=64, T=2, H=64, rows=1, dtype=2)
LINEAR = dict(x=1 << 20, x_scales=2 << 20, w=3 << 20, w_scales=4 << 20, out=5 << 20, xs=64, ws=64, os=40, M=2, N=40,
              K=64, out_dtype=2)
SAMPLE = dict(logits=1 << 20, uniforms=2 << 20, temperature=0, top_k=0, top_p=0, min_p=0, tokens=3 << 20, logprobs=0,
              stride=100, B=2, V=100, dtype=2)


def _quant(m, **kw):
    return m.library().moe_quantize_e4m3(m._QUANT_T.pack(*{**QUANT, **kw}.values()), None)


def _linear(m, work=4096, work_bytes=256, **kw):
    return m.library().moe_linear_e4m3(m._LINEAR_T.pack(*{**LINEAR, **kw}.values()), work, work_bytes, None)


def _sample(m, **kw):
    return m.library().moe_sample(m._SAMPLING_T.pack(*{**SAMPLE, **kw}.values()), None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(rows=0), 1), (dict(rows=2), 1), (dict(rows=64), 1), (dict(dtype=3), 2),
    (dict(dtype=4), 2), (dict(x=0), 1), (dict(out=0), 1), (dict(scales=0), 1), (dict(xs=63), 1), (dict(os=63), 1),
    (dict(x=(1 << 20) + 1), 1), (dict(scales=(3 << 20) + 2), 1), (dict(out=(1 << 20) + 255), 1),
    (dict(scales=(1 << 20) + 128), 1), (dict(scales=(2 << 20) + 64), 1), (dict(xs=1 << 62), 1),
    (dict(T=2 ** 31 - 1, H=256, xs=256, os=256, x=1 << 50, out=1 << 52), 2),
])
def test_quantize_refusals(m, change, code):
    assert _quant(m, **change) == code, m.moe_last_error()
    assert m.moe_last_error() != ""


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=0), 1), (dict(out_dtype=4), 2), (dict(out_dtype=0), 2), (dict(x=0), 1),
    (dict(x_scales=0), 1), (dict(w=0), 1), (dict(w_scales=0), 1), (dict(out=0), 1), (dict(work=0), 3),
    (dict(work=4112), 3), (dict(work_bytes=255), 3), (dict(xs=48), 1), (dict(ws=48), 1), (dict(os=39), 1),
    (dict(x=(1 << 20) + 8), 2), (dict(w=(3 << 20) + 1), 2), (dict(xs=72), 2), (dict(ws=65), 2),
    (dict(out=(5 << 20) + 1), 1), (dict(out=(5 << 20) + 2, out_dtype=3), 1), (dict(x_scales=(2 << 20) + 2), 1),
    (dict(out=(1 << 20) + 64), 1), (dict(out=(3 << 20) + 64), 1), (dict(out=2 << 20), 1), (dict(out=4 << 20), 1),
    (dict(out=4096), 1), (dict(xs=1 << 62), 1), (dict(xs=1 << 45, x=1 << 50), 1),
    (dict(M=2 ** 31 - 1, N=2 ** 31 - 1, os=2 ** 31), 2),
])
def test_linear_refusals(m, change, code):
    assert _linear(m, **change) == code, m.moe_last_error()
    assert m.moe_last_error() != ""


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), 1), (dict(V=0), 1), (dict(V=393217, stride=393217), 2), (dict(B=2 ** 24 + 1), 2), (dict(dtype=4), 2),
    (dict(logits=0), 1), (dict(uniforms=0), 1), (dict(tokens=0), 1), (dict(stride=99), 1), (dict(stride=1 << 62), 1),
    (dict(logits=(1 << 20) + 1), 1), (dict(logits=(1 << 20) + 2, dtype=3), 1), (dict(tokens=(3 << 20) + 4), 1),
    (dict(uniforms=(2 << 20) + 2), 1), (dict(logprobs=(4 << 20) + 1), 1), (dict(top_k=(4 << 20) + 1), 1),
    (dict(tokens=(1 << 20) + 8), 1), (dict(tokens=2 << 20), 1), (dict(logprobs=(3 << 20) + 8), 1),
    (dict(logprobs=2 << 20), 1), (dict(tokens=4 << 20, min_p=(4 << 20) + 8), 1),
])
def test_sample_refusals(m, change, code):
    assert _sample(m, **change) == code, m.moe_last_error()
    assert m.moe_last_error() != ""


def test_without_rows_nothing_runs(m):
    lib = m.library()
    assert _quant(m, T=0, x=0, out=0, scales=0) == 0
    assert _linear(m, M=0, x=0, x_scales=0, out=0) == 0
    assert _linear(m, N=0, w=0, w_scales=0, out=0) == 0
    assert _sample(m, B=0, logits=0, uniforms=0, tokens=0) == 0
    assert lib.moe_quantize_e4m3(None, None) == 1
    assert lib.moe_linear_e4m3(None, 4096, 256, None) == 1
    assert lib.moe_sample(None, None) == 1


def test_packed_structs_have_the_headers_layout(m):
    assert m._QUANT_T.size == 3 * 8 + 2 * 8 + 4 * 4
    assert m._LINEAR_T.size == 5 * 8 + 3 * 8 + 4 * 4
    assert m._SAMPLING_T.size == 8 * 8 + 8 + 3 * 4 + 4


def test_binding_refuses_before_the_library(m):
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    x, q, s = torch.zeros(3, 256, dtype=bf), torch.zeros(3, 256).to(e4), torch.zeros(3, 2)
    w, ws = torch.zeros(200, 256).to(e4), torch.zeros(2, 2)
    out, work = torch.zeros(3, 200), torch.zeros(256, dtype=torch.uint8)
    l, u, t = torch.zeros(3, 50), torch.zeros(3), torch.zeros(3, dtype=torch.int64)
    bad = [
        lambda: m.moe_quantize_e4m3(x, q, s),  # not on a GPU
        lambda: m.moe_quantize_e4m3(x.float(), q, s),
        lambda: m.moe_quantize_e4m3(x[0], q[0], s[0]),
        lambda: m.moe_quantize_e4m3(x, x, s),
        lambda: m.moe_quantize_e4m3(x, q[:2], s),
        lambda: m.moe_quantize_e4m3(x, q, s[:, :1]),
        lambda: m.moe_quantize_e4m3(x, q, s, rows=128),
        lambda: m.moe_quantize_e4m3(x, q, s[:1], rows=64),
        lambda: m.moe_quantize_e4m3(x, q, s, rows=1.5),
        lambda: m.moe_quantize_e4m3(x, q, s.double()),
        lambda: m.moe_quantize_e4m3(x, None, s),
        lambda: m.moe_quantize_e4m3(x.t().contiguous().t(), q, s),
        lambda: m.moe_linear_e4m3(q, s, w, ws, out, work),  # not on a GPU
        lambda: m.moe_linear_e4m3(x, s, w, ws, out, work),
        lambda: m.moe_linear_e4m3(q, s, w[:, :128], ws, out, work),
        lambda: m.moe_linear_e4m3(q, s, w, ws[:1], out, work),
        lambda: m.moe_linear_e4m3(q, s[:, :1], w, ws, out, work),
        lambda: m.moe_linear_e4m3(q, s, w, ws, out.double(), work),
        lambda: m.moe_linear_e4m3(q, s, w, ws, out[:, :199], work),
        lambda: m.moe_linear_e4m3(q, s, w, ws, out, None),
        lambda: m.moe_linear_e4m3(q[0], s[0], w, ws, out[0], work),
        lambda: m.moe_linear_e4m3(q, None, w, ws, out, work),
        lambda: m.moe_sample(l, u, t),  # not on a GPU
        lambda: m.moe_sample(l[0], u, t),
        lambda: m.moe_sample(l[:, :0], u, t),
        lambda: m.moe_sample(l.double(), u, t),
        lambda: m.moe_sample(l.t().contiguous().t(), u, t),
        lambda: m.moe_sample(l, u[:2], t),
        lambda: m.moe_sample(l, u, t.int()),
        lambda: m.moe_sample(l, u, t, temperature=0.7),
        lambda: m.moe_sample(l, u, t, top_k=t),
        lambda: m.moe_sample(l, u, t, logprobs=u.double()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")

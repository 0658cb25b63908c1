"""The compiled and the Python form of the checks of the quantisation, the 8-bit
product and the drawing of tokens make the same calls and refuse the same arguments."""
import pytest
import torch

from tests.test_gpu_fast_call import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture
def forms(m, monkeypatch):  # noqa: F811
    def each():
        for f in (m._fast_projections, None):
            monkeypatch.setattr(m, "_fast_projections", f)
            yield
    assert m._fast_projections is not None
    return each


def test_both_forms_make_the_same_calls(m, forms):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(5, 320, generator=g, device=DEV).to(torch.bfloat16)[:, :272]
    w = torch.randn(200, 272, generator=g, device=DEV).to(torch.float16)
    u = torch.rand(5, generator=g, device=DEV)
    t, p, k = torch.full((5,), 0.8, device=DEV), torch.full((5,), 0.9, device=DEV), torch.full((5,), 30, device=DEV).int()
    ws = m.alloc_status_workspace(DEV)
    side = torch.cuda.Stream()
    results = []
    for _ in forms():
        for st in (None, side, side.cuda_stream):
            torch.cuda.synchronize()
            q, s = torch.empty(5, 288, device=DEV, dtype=E4)[:, :272], torch.empty(5, 3, device=DEV)
            wq, wsc = torch.empty(200, 272, device=DEV, dtype=E4), torch.empty(2, 3, device=DEV)
            torch.cuda.synchronize()
            m.moe_quantize_e4m3(x, q, s, stream=st)
            m.moe_quantize_e4m3(w, wq, wsc, rows=128, stream=st)
            outs = [torch.empty(5, 210, device=DEV, dtype=d)[:, :200] for d in (torch.float32, torch.bfloat16, torch.float16)]
            torch.cuda.synchronize()
            for o in outs:
                m.moe_linear_e4m3(q, s, wq, wsc, o, ws, stream=st)
            tok = [torch.empty(5, dtype=torch.int64, device=DEV) for _ in range(3)]
            lp = torch.empty(5, device=DEV)
            torch.cuda.synchronize()
            for o, n in zip(outs, tok):
                m.moe_sample(o, u, n, temperature=t, top_k=k, top_p=p, min_p=t * 0.01, logprobs=lp, stream=st)
            m.moe_sample(outs[0], u, tok[1], stream=st)
            torch.cuda.synchronize()
            results.append([q.float(), s, wq.float(), wsc, *outs, *tok, lp])
    for r in results[1:]:
        for a, b in zip(results[0], r):
            assert torch.equal(a, b)


def test_both_forms_refuse_the_same_arguments(m, forms):  # noqa: F811
    x = torch.ones(3, 256, dtype=torch.bfloat16, device=DEV)
    q, s = torch.zeros(3, 256, device=DEV).to(E4), torch.ones(3, 2, device=DEV)
    w, wsc = torch.zeros(200, 256, device=DEV).to(E4), torch.ones(2, 2, device=DEV)
    out, ws = torch.zeros(3, 200, device=DEV), m.alloc_status_workspace(DEV)
    u, tok = torch.zeros(3, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    bad = [
        lambda: m.moe_quantize_e4m3(x.float(), q, s), lambda: m.moe_quantize_e4m3(x, q, s.cpu()),
        lambda: m.moe_quantize_e4m3(x, q, s, rows=128), lambda: m.moe_quantize_e4m3(x, q, s, rows=7),
        lambda: m.moe_quantize_e4m3(x, q, s, rows=None), lambda: m.moe_quantize_e4m3(x, q[:, :128], s),
        lambda: m.moe_quantize_e4m3(x.t().contiguous().t(), q, s), lambda: m.moe_quantize_e4m3(None, q, s),
        lambda: m.moe_linear_e4m3(x, s, w, wsc, out, ws), lambda: m.moe_linear_e4m3(q, s, w.cpu(), wsc, out, ws),
        lambda: m.moe_linear_e4m3(q, s, w, wsc.t(), out, ws), lambda: m.moe_linear_e4m3(q, s, w, wsc, out.double(), ws),
        lambda: m.moe_linear_e4m3(q, s, w, wsc, out, ws.cpu()), lambda: m.moe_linear_e4m3(q, s, w, wsc, out, ws[::2]),
        lambda: m.moe_linear_e4m3(q, s, w, wsc, out, ws[:1].expand(512)), lambda: m.moe_linear_e4m3(q, s, w, None, out, ws),
        lambda: m.moe_linear_e4m3(q, s[:2], w, wsc, out, ws), lambda: m.moe_linear_e4m3(q, s, w, wsc, out, 3),
        lambda: m.moe_sample(out.double(), u, tok), lambda: m.moe_sample(out, u.cpu(), tok),
        lambda: m.moe_sample(out, u, tok.int()), lambda: m.moe_sample(out, u, tok, temperature=1.0),
        lambda: m.moe_sample(out, u, tok, top_k=tok), lambda: m.moe_sample(out, u, tok, logprobs=u[:2]),
        lambda: m.moe_sample(out[:, :0], u, tok), lambda: m.moe_sample(out, None, tok),
    ]
    library = [
        lambda: m.moe_linear_e4m3(q[:, 8:136], s[:, :1].contiguous(), w[:, :128], wsc[:, :1].contiguous(), out, ws),
        lambda: m.moe_linear_e4m3(q, s, w, wsc, out, ws[:128]),
        lambda: m.moe_linear_e4m3(q, s, w, wsc, out[:1].expand(3, 200), ws),
        lambda: m.moe_sample(torch.zeros(3, 393217, device=DEV), u, tok),
        lambda: m.moe_sample(out, u, tok, logprobs=u),
        lambda: m.moe_quantize_e4m3(x, x.view(E4)[:, :256], s),
    ]
    for _ in forms():
        for i, call in enumerate(bad):
            with pytest.raises(ValueError):
                call()
                pytest.fail(f"call {i} was taken")
        for i, call in enumerate(library):
            with pytest.raises(m.MoeError):
                call()
                pytest.fail(f"call {i} was taken")

"""The compiled and the Python form of the layer operators' checks make the same
calls and refuse the same arguments."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    mod.library()
    if mod._fast is None:
        pytest.skip("fast_call.cpp is not built here")
    return mod


def _calls(m):
    g = torch.Generator(device=DEV).manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    x, r, w = rn(5, 192)[:, :128], rn(5, 128), rn(128)
    k, v = (torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = m.MoeKvCache(k, v)
    ws = m.alloc_attention_workspace(cache, 8)
    qkv = rn(5, 12 * 64)
    q, kn, vn = qkv[:, :512].unflatten(1, (8, 64)), qkv[:, 512:640].unflatten(1, (2, 64)), qkv[:, 640:].unflatten(1, (2, 64))
    pos, slots = torch.arange(5, device=DEV) + 7, torch.arange(5, device=DEV) * 17
    freq, qw = torch.rand(16, generator=g, device=DEV), rn(64)
    table = torch.arange(5, dtype=torch.int32, device=DEV)[:, None].contiguous()
    lens = torch.tensor([3, 0, 16, 9, 5], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()

    def norm(stream=None, **kw):
        o, ro = torch.empty(5, 128, dtype=torch.bfloat16, device=DEV), torch.empty_like(r)
        m.moe_add_rmsnorm(x, w, o, residual=r, residual_out=ro, eps=1e-5, stream=stream)
        q8, s = torch.empty(5, 128, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(5, 2, device=DEV)
        m.moe_add_rmsnorm(x, w, q8, scales=s, group=64, stream=stream)
        return o, ro, q8.float(), s

    def rope(stream=None):
        k.zero_(), v.zero_()
        o = torch.empty(5, 8, 64, dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        m.moe_rope_append(cache, q, kn, vn, pos, slots, freq, o, ws, q_norm_w=qw, k_norm_w=qw, eps=1e-5,
                          interleaved=True, stream=stream)
        torch.cuda.synchronize()
        return o, k.clone(), v.clone()

    def attention(stream=None):
        o, lse = torch.empty(5, 8, 64, dtype=torch.bfloat16, device=DEV), torch.empty(5, 8, device=DEV)
        m.moe_paged_attention(cache, q, table, lens, o, ws, scale=0.2, window=7, lse=lse, stream=stream)
        o2 = torch.empty_like(o)
        m.moe_paged_attention(cache, q, table, lens, o2, ws, stream=stream)
        return o, lse, o2

    return (norm, rope, attention), side


def test_both_forms_make_the_same_calls(m, monkeypatch):
    calls, side = _calls(m)
    for call in calls:
        streams = [None, side, side.cuda_stream]
        results = []
        for fast in (m._fast, None):
            monkeypatch.setattr(m, "_fast", fast)
            for st in streams:
                torch.cuda.synchronize()
                out = call(stream=st)
                torch.cuda.synchronize()
                results.append(out)
        monkeypatch.undo()
        for out in results[1:]:
            for a, b in zip(results[0], out):
                assert torch.equal(a, b)


def test_both_forms_refuse_the_same_arguments(m, monkeypatch):
    x, w = torch.ones(2, 64, dtype=torch.bfloat16, device=DEV), torch.ones(64, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    cache = m.MoeKvCache(kv, kv.clone())
    ws = m.alloc_attention_workspace(cache, 4)
    q, k = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos, f = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(16, device=DEV)
    table, lens = torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    e4 = torch.zeros(2, 64, dtype=torch.float8_e4m3fn, device=DEV)
    bad = [
        lambda: m.moe_add_rmsnorm(x, w.cpu(), x),
        lambda: m.moe_add_rmsnorm(x, w, x[:, :32]),
        lambda: m.moe_add_rmsnorm(x, w, x.half()),
        lambda: m.moe_add_rmsnorm(x, w, e4),
        lambda: m.moe_add_rmsnorm(x, w, e4, scales=torch.zeros(2, 1)),
        lambda: m.moe_add_rmsnorm(x, w, x, residual=x.t().contiguous().t()),
        lambda: m.moe_add_rmsnorm(x, w, x, residual_out=x),
        lambda: m.moe_rope_append(cache, q, k, k, pos.int(), pos, f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos.cpu(), f, q, ws),
        lambda: m.moe_rope_append(cache, q, k[:, :1], k, pos, pos, f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q, ws, q_norm_w=w),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q, ws.cpu()),
        lambda: m.moe_paged_attention(cache, q, table.long(), lens, q, ws),
        lambda: m.moe_paged_attention(cache, q, table, lens[:1], q, ws),
        lambda: m.moe_paged_attention(cache, q, table, lens, q.half(), ws),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, ws, lse=torch.zeros(2, 4)),
    ]
    library = [
        lambda: m.moe_add_rmsnorm(x, w, x, eps=-1.0),
        lambda: m.moe_add_rmsnorm(x, w, e4, scales=torch.zeros(2, 2, device=DEV), group=48),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f[:5], q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q, ws[:128]),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, ws[:4096]),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, ws, window=-1),
    ]
    for fast in (m._fast, None):
        monkeypatch.setattr(m, "_fast", fast)
        for call in bad:
            with pytest.raises(ValueError):
                call()
        for call in library:
            with pytest.raises(m.MoeError):
                call()

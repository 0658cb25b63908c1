"""Workspaces as the compiled and the Python form of the layer operators take them."""
import pytest
import torch

from tests.test_gpu_fast_call import DEV, m  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("fast", [True, False])
def test_workspaces(m, monkeypatch, fast):  # noqa: F811
    monkeypatch.setattr(m, "_fast", m._fast if fast else None)
    kv = torch.zeros(4, 16, 2, 64, dtype=BF, device=DEV)
    cache = m.MoeKvCache(kv, kv.clone())
    ws = m.alloc_attention_workspace(cache, 4)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k = (torch.randn(2, h, 64, generator=g, device=DEV).to(BF) for h in (4, 2))
    pos, f = torch.arange(2, device=DEV), torch.rand(32, device=DEV)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1, 1], dtype=torch.int32, device=DEV)

    def both(ws):
        qo, out = torch.zeros_like(q), torch.zeros_like(q)
        m.moe_rope_append(cache, q, k, k, pos, pos * 16, f, qo, ws)
        m.moe_paged_attention(cache, qo, table, lens, out, ws)
        torch.cuda.synchronize()
        return out

    want = both(ws)
    assert torch.equal(want, k.repeat_interleave(2, 1))  # one token: its value
    # the bytes count, whatever the elements are
    wide = torch.zeros(ws.numel() // 4 + 64, dtype=torch.float32, device=DEV)
    wide = wide[(-wide.data_ptr()) % 256 // 4:][:ws.numel() // 4]
    assert torch.equal(both(wide), want)
    m.moe_query_status(wide)
    for bad in (torch.zeros(1, dtype=torch.uint8, device=DEV).expand(ws.numel()),
                torch.zeros(2 * ws.numel(), dtype=torch.uint8, device=DEV)[::2]):
        for call in (lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q.clone(), bad),
                     lambda: m.moe_paged_attention(cache, q, table, lens, q.clone(), bad)):
            with pytest.raises(ValueError, match="ws"):
                call()
    for short in (wide[:32], ws[:128]):
        with pytest.raises(m.MoeError):
            m.moe_rope_append(cache, q, k, k, pos, pos, f, q.clone(), short)


@pytest.mark.parametrize("fast", [True, False])
def test_both_forms_refuse_what_no_argument_holds(m, monkeypatch, fast):  # noqa: F811
    monkeypatch.setattr(m, "_fast", m._fast if fast else None)
    x, w = torch.ones(2, 64, dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV)
    kv = torch.zeros(4, 16, 2, 64, dtype=BF, device=DEV)
    cache = m.MoeKvCache(kv, kv.clone())
    ws = m.alloc_attention_workspace(cache, 4)
    q, k = torch.zeros(2, 4, 64, dtype=BF, device=DEV), torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    pos, f = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(16, device=DEV)
    table, lens = torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    bad = [
        lambda: m.moe_add_rmsnorm(x, None, x),
        lambda: m.moe_add_rmsnorm(x, w, x, residual=2),
        lambda: m.moe_add_rmsnorm(x, w, x, eps=1e39),
        lambda: m.moe_add_rmsnorm(x, w, x, eps="1"),
        lambda: m.moe_rope_append(None, q, k, k, pos, pos, f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, None, f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q, ws, eps=1e39),
        lambda: m.moe_paged_attention(kv, q, table, lens, q, ws),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, None),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, ws, scale=1e39),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, ws, window=2 ** 31),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    m.moe_paged_attention(cache, q, table, lens, q.clone(), ws, scale=torch.tensor(0.25), window=2 ** 31 - 1)
    m.moe_query_status(ws)

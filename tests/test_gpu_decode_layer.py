"""The decoder layers of decode_layer.py, step by step: the attention half
against its 64-bit form on the stored inputs of each step, the block against
moe_grouped_forward on the same rows, eager steps against a captured graph."""
import pytest
import torch

from tests._layer_ref import F64, attention_ref, norm_ref, rope_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


def _cfg(m, **kw):
    from moe_decode_expert_gb300.decode_layer import LayerCfg
    return LayerCfg(m.MoeCfg(256, 16, 2, 64, 64, m.MOE_BF16, has_shared_gate=1), 8, 2, 64, 32, **kw)


def _rel(got, ref):
    return float((got.cpu().double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("kw", [dict(), dict(cache_e4m3=True, page_size=7), dict(window=3)])
def test_steps_match_the_plain_layer(m, kw):
    from moe_decode_expert_gb300 import decode_layer as dl
    cfg = _cfg(m, **kw)
    g = torch.Generator(device=DEV).manual_seed(1)
    layers = [dl.random_layer(cfg, DEV, g) for _ in range(2)]
    B, D, hq, hkv = 5, 64, 8, 2
    d = dl.Decoder(cfg, layers, B, 24, DEV)
    d.positions.copy_(torch.tensor([0, 1, 2, 9, 5]))  # earlier slots hold zeros
    steps = []
    attend = d.attend

    def watch(w, cache, qkv, slots, lens):
        out = attend(w, cache, qkv, slots, lens)
        steps.append((w, cache, qkv.cpu(), d.positions.cpu().clone(), lens.cpu(), cache.k.float().cpu(),
                      cache.v.float().cpu(), d.q.cpu().clone(), d.attn.cpu().clone()))
        return out

    d.attend = watch
    for _ in range(3):
        h = torch.randn(B, 256, generator=g, device=DEV).to(torch.bfloat16)
        before = len(steps)
        x, r = d.step(h)
        # the last layer's block again, by itself, on the rows it got
        w = layers[-1]
        again = torch.empty_like(x)
        m.moe_grouped_forward(cfg.moe, d.y, w["router_w"], w["w13"], w["w2"], w["shared_w13"], w["shared_w2"],
                              w["shared_gate_w"], d.ids, d.weights, again, d.ws_moe)
        assert torch.equal(again, x)
        # the first layer's projection: one rounding of y, one of the product
        first = steps[before]
        y = norm_ref(h.cpu(), layers[0]["norm1"].cpu(), None, cfg.eps)
        qkv = y @ layers[0]["qkv"].cpu().to(F64).t()
        assert _rel(first[2], qkv) <= 2.0 ** -8
        # the norm before the last block, from the residual it left
        yn = norm_ref(d.r.cpu(), w["norm2"].cpu(), None, cfg.eps)
        assert _rel(d.y, yn) <= 2.0 ** -7  # r was rounded once more than y's input
    d.check()
    for w, cache, qkv, pos, lens, k, v, q, attn in steps:
        qr, kr = qkv[:, :hq * D].view(B, hq, D), qkv[:, hq * D:(hq + hkv) * D].view(B, hkv, D)
        freq = d.inv_freq.cpu()
        qref, _ = rope_ref(qr, w["q_norm"].cpu(), pos, freq, cfg.eps, False)
        kref, _ = rope_ref(kr, w["k_norm"].cpu(), pos, freq, cfg.eps, False)
        assert _rel(q, qref) <= 2.0 ** -8
        s = 0.05 if cfg.cache_e4m3 else 1.0
        P = cfg.page_size
        table = d.block_table.cpu()
        page = table.gather(1, (pos // P)[:, None])[:, 0].long()
        got = k[page, pos % P].double() * s
        assert float((got - kref).norm() / kref.norm()) <= (2.0 ** -4 if cfg.cache_e4m3 else 2.0 ** -8)
        sc = torch.full((hkv,), 0.05) if cfg.cache_e4m3 else None
        ref, _, _, _ = attention_ref(q, k, v, table, lens, D ** -0.5, cfg.window, sc, sc, 0.0)
        assert _rel(attn, ref) <= 2.0 ** -8


def test_a_captured_step_equals_eager_steps(m):
    from moe_decode_expert_gb300 import decode_layer as dl
    cfg = _cfg(m)
    g = torch.Generator(device=DEV).manual_seed(2)
    layers = [dl.random_layer(cfg, DEV, g) for _ in range(2)]
    torch.manual_seed(0)
    h = torch.randn(3, 256, generator=g, device=DEV).to(torch.bfloat16)
    eager = dl.Decoder(cfg, layers, 3, 64, DEV)
    d = dl.Decoder(cfg, layers, 3, 64, DEV)
    want = [[t.clone() for t in eager.step(h)] for _ in range(6)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step(h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d.step(h)
    for i in range(1, 6):
        graph.replay()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
    d.check()

"""A decoder from token to token with 8-bit projections: every step's norm,
quantisations, products, attention and draw against their 64-bit forms on the stored
inputs, and eager steps against a captured graph."""
import pytest
import torch

from tests._layer_ref import F64, attention_ref, norm_ref
from tests._projection_ref import linear_ref, quant_ref, sample_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
V = 1003


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


def _decoder(m, B, **kw):
    from moe_decode_expert_gb300 import decode_layer as dl
    cfg = dl.LayerCfg(m.MoeCfg(272, 16, 2, 64, 64, m.MOE_BF16, has_shared_gate=1), 6, 2, 72, 32, linear_e4m3=True, **kw)
    g = torch.Generator(device=DEV).manual_seed(1)
    layers = [dl.random_layer(cfg, DEV, g) for _ in range(2)]
    head = dl.random_head(cfg, V, DEV, g)
    torch.manual_seed(0)
    return dl.Decoder(cfg, layers, B, 24, DEV, head), cfg, layers, head


def _same_product(out, a):
    ref, mag = linear_ref(*(t.cpu() for t in a))
    err = (out.cpu().double() - ref).abs()
    assert (err <= ref.abs() * (torch.finfo(out.dtype).eps / 2 + 2.0 ** -20) + mag * 2.0 ** -19).all()


def test_steps_match_their_plain_forms(m):
    B, D, hq, hkv = 5, 72, 6, 2
    d, cfg, layers, head = _decoder(m, B, page_size=7)
    seen = []
    attend = d.attend

    def watch(w, cache, qkv, slots, lens):
        y8, y8_s = d.y8.clone(), d.y8_s.clone()
        _same_product(qkv, (y8, y8_s, *w["qkv"]))
        out = attend(w, cache, qkv, slots, lens)
        ref, _, _, _ = attention_ref(d.q.cpu(), cache.k.cpu(), cache.v.cpu(), d.block_table.cpu(), lens.cpu(), D ** -0.5, 0,
                                     None, None, 0.0)
        assert float((d.attn.cpu().double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
        z, s = quant_ref(d.attn.view(B, hq * D).cpu(), 1)
        assert ((d.a8_s.cpu().double() - s).abs() <= s * 2.0 ** -24).all()
        tol = torch.maximum(z.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=F64)) * (1 + 2.0 ** -20)
        assert ((d.a8.float().cpu().double() - z).abs() <= tol).all()
        _same_product(out, (d.a8, d.a8_s, *w["o"]))
        seen.append((y8, y8_s))
        return out

    d.attend = watch
    g = torch.Generator().manual_seed(2)
    d.tokens.copy_(torch.randint(0, V, (B,), generator=g))
    asks = [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.0), (1.5, 0, 0.9, 0.01), (0.9, 0, 1.0, 0.1)]
    t, k, p, q = (torch.tensor([a[i] for a in asks], dtype=torch.int32 if i == 1 else torch.float32, device=DEV)
                  for i in range(4))
    asks = [(float(t[b]), int(k[b]), float(p[b]), float(q[b])) for b in range(B)]
    for _ in range(3):
        before, n = d.tokens.clone(), len(seen)
        u = torch.rand(B, generator=g)
        tokens = d.next_tokens(u.to(DEV), temperature=t, top_k=k, top_p=p, min_p=q)
        # the first layer's rows are the norm of the embedding's
        y = norm_ref(head["embed"][before].cpu(), layers[0]["norm1"].cpu(), None, cfg.eps)
        y8, s = seen[n]
        s = s.cpu().double().repeat_interleave(128, 1)[:, :272]
        assert ((y8.float().cpu().double() * s - y).abs() <= y.abs() * 2.0 ** -4 + s * 2.0 ** -9).all()
        # the last norm, from the residual that it left
        yn = norm_ref(d.r.cpu(), head["norm"].cpu(), None, cfg.eps)
        s = d.y8_s.cpu().double().repeat_interleave(128, 1)[:, :272]
        got = d.y8.float().cpu().double() * s
        assert float((got - yn).norm()) <= 2.0 ** -4 * float(yn.norm())
        _same_product(d.logits, (d.y8, d.y8_s, *head["out"]))
        for b in range(B):
            want = sample_ref(d.logits[b].cpu(), *asks[b], float(u[b]))
            assert want[2] <= 2.0 ** -26 or int(tokens[b]) == want[0]
            assert abs(float(d.logprobs[b]) - want[1]) <= 2.0 ** -20 * abs(want[1]) + 2.0 ** -27
    d.check()
    assert d.positions.tolist() == [3] * B


def test_a_captured_step_equals_eager_steps(m):
    eager, *_ = _decoder(m, 3)
    d, *_ = _decoder(m, 3)
    full = lambda v: torch.full((3,), v, device=DEV)  # noqa: E731
    u, asked = torch.zeros(3, device=DEV), dict(temperature=full(1.0), top_p=full(0.9))
    draws = torch.rand(6, 3, generator=torch.Generator().manual_seed(3)).to(DEV)
    want = []
    for i in range(6):
        u.copy_(draws[i])
        want.append(eager.next_tokens(u, **asked).clone())
    side = torch.cuda.Stream()
    u.copy_(draws[0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = d.next_tokens(u, **asked).clone()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.next_tokens(u, **asked)
    for i in range(1, 6):
        u.copy_(draws[i])
        graph.replay()
        assert torch.equal(d.tokens, want[i])
    assert torch.equal(d.logits, eager.logits)
    d.check()


def test_without_a_head_or_with_odd_sizes(m):
    from moe_decode_expert_gb300 import decode_layer as dl
    cfg = dl.LayerCfg(m.MoeCfg(264, 16, 2, 64, 64, m.MOE_BF16), 8, 2, 64, 32)
    layers = [dl.random_layer(cfg, DEV)]
    d = dl.Decoder(cfg, layers, 2, 16, DEV)
    with pytest.raises(ValueError):
        d.next_tokens(torch.zeros(2, device=DEV))
    with pytest.raises(ValueError):
        dl.Decoder(cfg, layers, 2, 16, DEV, dl.random_head(cfg, 64, DEV))

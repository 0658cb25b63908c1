"""Decoder steps at and past the last place of the table: other sequences go on, nothing
is stored, and check() raises."""
import pytest
import torch

from tests.test_gpu_decode_layer import DEV, _cfg, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_steps_past_the_table_are_reported(m, captured):  # noqa: F811
    from moe_decode_expert_gb300 import decode_layer as dl
    cfg = _cfg(m)
    g = torch.Generator(device=DEV).manual_seed(3)
    layers = [dl.random_layer(cfg, DEV, g) for _ in range(2)]
    h = torch.randn(3, 256, generator=g, device=DEV).to(torch.bfloat16)
    start = torch.tensor([2, 13, 0])  # 16 places: the second sequence has three steps left
    d = dl.Decoder(cfg, layers, 3, 16, DEV)
    assert d.max_len == 16
    step = lambda: d.step(h)  # noqa: E731
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            d.step(h)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d.step(h)
        step = graph.replay
        for c in d.caches:
            c.k.zero_(), c.v.zero_()
    d.positions.copy_(start)
    for _ in range(3):
        step()
    d.check()
    kept = [(c.k.clone(), c.v.clone()) for c in d.caches]
    others = d.block_table[[0, 2]].flatten().long()
    for _ in range(2):
        step()
        with pytest.raises(m.MoeError) as ei:
            d.check()
        assert ei.value.code == 6 and "length" in str(ei.value) and " 1" in str(ei.value)
    # the sequence past the end stored nothing more, the others did
    mine = d.block_table[1].long()
    for c, (k, v) in zip(d.caches, kept):
        assert torch.equal(c.k[mine], k[mine]) and torch.equal(c.v[mine], v[mine])
        assert not torch.equal(c.k[others], k[others])
    # and the others' results are those of a decoder in which it has room (but for last
    # places of bf16: the attention's work is split by all lengths)
    wide = dl.Decoder(cfg, layers, 3, 32, DEV)
    wide.positions.copy_(start)
    for _ in range(5):
        x, r = wide.step(h)
    wide.check()
    keep = [0, 2]
    for got, want in ((d.r[keep].double(), r[keep].double()), (d.x[keep].double(), x[keep].double())):
        assert (got - want).norm() <= 2.0 ** -7 * want.norm()
    assert torch.isfinite(d.x).all()

"""The layer operators' Python checks on CPU tensors: the first thing wrong is named."""
import pytest
import torch

from tests.test_layer_host import m  # noqa: F401

BF = torch.bfloat16


def _args(m, ws=None):  # noqa: F811
    kv = torch.zeros(4, 16, 2, 64, dtype=BF)
    cache = m.MoeKvCache(kv, kv.clone())
    ws = m.alloc_attention_workspace(cache, 4) if ws is None else ws
    q, k = torch.zeros(2, 4, 64, dtype=BF), torch.zeros(2, 2, 64, dtype=BF)
    pos, f = torch.zeros(2, dtype=torch.int64), torch.zeros(32)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    return ([cache, q, k, k, pos, pos, f, q, ws], [cache, q, table, lens, q.clone(), ws])


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 28),
                                torch.zeros(1 << 10, dtype=torch.uint8)[::2], [1, 2]])
def test_a_workspace_of_other_memory_than_it_counts_is_refused(m, ws):  # noqa: F811
    """A workspace's size is what its elements are, one after the other: an expanded
    tensor counts elements that share a byte of memory."""
    rope, attn = _args(m, ws)
    for call, args in ((m.moe_rope_append, rope), (m.moe_paged_attention, attn)):
        with pytest.raises(ValueError, match="ws"):
            call(*args)


def test_what_is_no_tensor_is_named(m):  # noqa: F811
    x, w = torch.zeros(2, 64, dtype=BF), torch.zeros(64, dtype=BF)
    for args, kw, name in (((None, w, x), {}, "x"), ((x, None, x), {}, "weight"), ((x, w, None), {}, "out"),
                           ((x, w, x), dict(residual=1.0), "residual"), ((x, w, x), dict(residual=x, residual_out=[]), "residual_out"),
                           ((x, w, x.to(torch.float8_e4m3fn)), dict(scales=3), "scales")):
        with pytest.raises(ValueError, match=rf"^{name}\b"):
            m.moe_add_rmsnorm(*args, **kw)
    rope, attn = _args(m)
    for call, args, names in ((m.moe_rope_append, rope, "cache q k v positions slots inv_freq q_out ws".split()),
                              (m.moe_paged_attention, attn, "cache q block_table seq_lens out ws".split())):
        for i, name in enumerate(names):
            with pytest.raises(ValueError, match=rf"^{name}\b"):
                call(*args[:i], None, *args[i + 1:])
    with pytest.raises(ValueError, match="^k_norm_w"):
        m.moe_rope_append(*rope, q_norm_w=torch.zeros(64, dtype=BF), k_norm_w=2)
    with pytest.raises(ValueError, match="^lse"):
        m.moe_paged_attention(*attn, lse=0)
    kv = torch.zeros(4, 16, 2, 64, dtype=BF)
    for k, v, s, name in ((None, kv, None, "k"), (kv, None, None, "v"), (kv.to(torch.float8_e4m3fn), kv, None, "v"),
                          (kv.to(torch.float8_e4m3fn), kv.to(torch.float8_e4m3fn), 1.0, "k_scale")):
        with pytest.raises(ValueError, match=rf"^{name}\b"):
            m.MoeKvCache(k, v, s, s)


def test_numbers_that_no_argument_holds_are_refused(m):  # noqa: F811
    x, w = torch.zeros(2, 64, dtype=BF), torch.zeros(64, dtype=BF)
    e4, s = x.to(torch.float8_e4m3fn), torch.zeros(2, 1)
    _, attn = _args(m)
    for call in (lambda: m.moe_add_rmsnorm(x, w, e4, scales=s, group=2 ** 40),
                 lambda: m.moe_add_rmsnorm(x, w, x, eps="small"),
                 lambda: m.moe_paged_attention(*attn, window=2 ** 31),
                 lambda: m.moe_paged_attention(*attn, window=None),
                 lambda: m.moe_paged_attention(*attn, window=1.5),
                 lambda: m.moe_paged_attention(*attn, scale="1")):
        with pytest.raises(ValueError, match="group|eps|window|scale"):
            call()


def test_numbers_past_fp32_are_refused(m):  # noqa: F811
    x, w = torch.zeros(2, 64, dtype=BF), torch.zeros(64, dtype=BF)
    rope, attn = _args(m)
    for call in (lambda: m.moe_add_rmsnorm(x, w, x, eps=1e39), lambda: m.moe_rope_append(*rope, eps=1e300),
                 lambda: m.moe_paged_attention(*attn, scale=-1e39)):
        with pytest.raises(ValueError, match="fp32"):
            call()

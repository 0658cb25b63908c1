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

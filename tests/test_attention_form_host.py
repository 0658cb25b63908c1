"""Which kernels serve which batches, asked on the host."""
import pytest
import torch

from tests.test_layer_host import m  # noqa: F401


def _cache(m, hkv, D, dtype=torch.bfloat16, page=16):  # noqa: F811
    kv = torch.zeros(1, page, hkv, D, dtype=dtype)
    return m.MoeKvCache(kv, kv)


@pytest.mark.parametrize("B,hkv,pages,window,form", [
    (1, 2, 1 << 20, 0, "teams"), (2, 2, 1 << 20, 0, "teams"), (3, 2, 1 << 20, 0, "ctas"), (16, 2, 64, 0, "teams"),
    (17, 2, 64, 0, "ctas"), (16, 2, 1 << 20, 0, "ctas"), (16, 2, 1 << 20, 500, "teams"), (64, 2, 4, 0, "ctas")])
def test_form(m, B, hkv, pages, window, form):  # noqa: F811
    assert m.moe_attention_form(_cache(m, hkv, 256), B, 8 * hkv, pages, window) == form


def test_refused_sizes_have_none(m):  # noqa: F811
    c = _cache(m, 2, 128)
    for args in ((0, 4, 1), (-1, 4, 1), (1, 3, 1), (1, 0, 1), (1, 4, -1), (1, 4, 1, -1)):
        assert m.moe_attention_form(c, *args) is None
    assert m.library().moe_attention_form(None, 1, 4, 1, 0) == 0

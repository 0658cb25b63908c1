"""The limit that the header states for a batch's places is the one that is kept."""
import os
import re

import pytest
import torch

from tests.test_layer_host import _attn, m  # noqa: F401

# (what is within the limit goes on to a launch with made-up addresses, so it has to find no GPU)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls with made-up addresses")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")


def _stated():
    text = re.sub(r"\s*\n \*\s*", " ", open(HEADER).read())
    mt = re.search(r"Limits: (.*?) below 2\^31", text)
    return eval("lambda B, n_kv_heads, n_q_heads, max_pages, page_size: " +  # noqa: S307
                mt.group(1).replace("ceil(n_q_heads / n_kv_heads / 8)", "-(-n_q_heads // n_kv_heads // 8)")
                .replace("/ 16", "// 16"))


@pytest.mark.parametrize("hkv,group", [(4, 1), (4, 8), (4, 9), (1, 16), (1, 17), (2, 64)])
def test_the_stated_limit(m, hkv, group):  # noqa: F811
    stated, page = _stated(), 16
    for B in (1, 7, 1000):
        kw = dict(B=B, n_kv_heads=hkv, hq=hkv * group, page_size=page)
        lo, hi = 1, 2 ** 31 - 1  # the largest number of pages within what is stated
        while lo < hi:
            mid = (lo + hi + 1) // 2
            lo, hi = (mid, hi) if stated(B, hkv, hkv * group, mid, page) < 2 ** 31 else (lo, mid - 1)
        if lo < 2 ** 31 - 1:
            assert _attn(m, **kw, max_pages=lo + 1) == 2, m.moe_last_error()
        assert _attn(m, **kw, max_pages=lo) not in (0, 1, 2, 3), m.moe_last_error()

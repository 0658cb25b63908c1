"""The attention's workspace holds what a launch can write: per chunk of the line two
slots, per CTA three chunks (its own and two small ones), up to 160 SMs."""
import pytest
import torch

from tests.test_layer_host import CACHE, m  # noqa: F401


@pytest.mark.parametrize("group", [1, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("D", [8, 64, 72, 128, 136, 256])
def test_every_slot_has_its_place(m, D, group):  # noqa: F811
    hkv = CACHE["n_kv_heads"]
    got = m.library().moe_attention_workspace_bytes(m._CACHE_T.pack(*{**CACHE, "head_dim": D}.values()), hkv * group)
    dp = 64 if D <= 64 else 128 if D <= 128 else 256  # columns of a slot
    ctas = 4 if dp == 64 else 2                        # of an SM
    heads = 16 if group > 8 and dp < 256 else 8        # of a slot
    chunks = 3 * 160 * ctas
    slots = 2 * chunks
    outputs, statistics, counters = slots * heads * dp * 4, slots * 16 * 8, chunks * 4 * 4
    assert got >= 256 + counters + 256 + statistics + outputs and got % 256 == 0


def test_teams_fit_too(m):  # noqa: F811
    """Forty teams at most, two slots each, and a copy of the statistics per rank."""
    for D in (64, 128, 256):
        got = m.library().moe_attention_workspace_bytes(m._CACHE_T.pack(*{**CACHE, "head_dim": D}.values()), 4)
        assert got >= 256 + 40 * 8 * 4 + 80 * 8 * 16 * 8 + 80 * 8 * D * 4


def test_a_smaller_workspace_is_refused(m):  # noqa: F811
    from tests.test_layer_host import _attn
    if torch.cuda.is_available():
        pytest.skip("calls with made-up addresses")
    for D in (64, 128, 256):
        for hq in (4, 40):
            n = m.library().moe_attention_workspace_bytes(m._CACHE_T.pack(*{**CACHE, "head_dim": D}.values()), hq)
            kw = dict(head_dim=D, hq=hq, kp=1 << 16, kt=1 << 12, kh=D, vp=1 << 16, vt=1 << 12, vh=D)
            assert _attn(m, ws_bytes=n - 1, **kw) == 3 and _attn(m, ws_bytes=n, **kw) not in (0, 1, 2, 3)

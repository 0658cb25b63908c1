"""Host-side checks of the layer operators (norm, rotation + append, paged
attention): every refusal of the C entries and of the binding, before anything
touches a GPU."""
import ctypes
import struct

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


NORM = dict(x=256, residual=512, weight=768, out=1024, residual_out=512, scales=0, xs=64, rs=64, os=64, ros=64, T=2,
            H=64, dtype=2, out_dtype=2, group=0, eps=1e-6)


def _norm(m, **kw):
    a = {**NORM, **kw}
    return m.library().moe_add_rmsnorm(m._NORM_T.pack(*a.values()), None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=32769, xs=32769, rs=32769, os=32769, ros=32769), 2),
    (dict(dtype=3), 2), (dict(out_dtype=1), 2), (dict(out_dtype=3), 2), (dict(x=0), 1), (dict(weight=0), 1),
    (dict(out=0), 1), (dict(residual=0), 1), (dict(out_dtype=4), 1), (dict(scales=2048), 1), (dict(group=64), 1),
    (dict(out_dtype=4, scales=2048, group=48), 1), (dict(out_dtype=4, scales=2048, group=8), 1),
    (dict(out_dtype=4, scales=2048, group=512), 1), (dict(out_dtype=4, scales=2050), 1), (dict(x=257), 1),
    (dict(xs=63), 1), (dict(ros=63), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(out_dtype=4, scales=2048, group=64, x=258), 2), (dict(out_dtype=4, scales=2048, group=64, xs=65), 2),
    (dict(out_dtype=4, scales=2048, group=32, H=63), 2),
])
def test_norm_refusals(m, change, code):
    assert _norm(m, **change) == code, m.moe_last_error()
    assert m.moe_last_error() != ""


def test_norm_without_rows_is_a_no_op(m):
    assert _norm(m, T=0, x=0, residual=0, weight=0, out=0, residual_out=0) == 0
    assert m.library().moe_add_rmsnorm(None, None) == 1


CACHE = dict(k=256, v=512, k_scale=0, v_scale=0, kp=8192, kt=512, kh=128, vp=8192, vt=512, vh=128, n_pages=4,
             page_size=16, n_kv_heads=4, head_dim=128, dtype=2)
ROPE = dict(q=256, k=512, v=768, q_out=1024, positions=2048, slots=4096, inv_freq=8192, qn=0, kn=0, qt=1024, qh=128,
            kt=512, kh=128, vt=512, vh=128, ot=1024, oh=128, T=2, hq=8, rot=64, dtype=2, interleaved=0, eps=1e-6)
ATTN = dict(q=256, out=512, lse=0, table=1024, lens=2048, qs=1024, qh=128, os=1024, oh=128, ts=8, B=2, hq=8,
            max_pages=8, window=0, dtype=2, scale=0.1)


def _cache(m, kw):
    return m._CACHE_T.pack(*{**CACHE, **{n: kw.pop(n) for n in list(kw) if n in CACHE and n not in ("k", "v", "dtype")},
                             **{n[6:]: kw.pop(n) for n in list(kw) if n.startswith("cache_")}}.values())


def _rope(m, ws=4096, ws_bytes=1 << 26, **kw):
    c = _cache(m, kw)
    return m.library().moe_rope_append(c, m._ROPE_T.pack(*{**ROPE, **kw}.values()), ws, ws_bytes, None)


def _attn(m, ws=4096, ws_bytes=1 << 26, **kw):
    c = _cache(m, kw)
    return m.library().moe_paged_attention(c, m._ATTN_T.pack(*{**ATTN, **kw}.values()), ws, ws_bytes, None)


CACHE_REFUSALS = [
    (dict(n_pages=0), 1), (dict(page_size=0), 1), (dict(n_kv_heads=0), 1), (dict(head_dim=0), 1),
    (dict(head_dim=100), 2), (dict(head_dim=264), 2), (dict(cache_dtype=1), 2), (dict(cache_dtype=3), 2),
    (dict(cache_dtype=4, head_dim=72), 2), (dict(cache_k=0), 1), (dict(cache_v=264), 1), (dict(kp=8196), 2),
    (dict(vt=516), 2), (dict(vp=-8192), 2), (dict(kp=(1 << 30) + 8), 2), (dict(k_scale=64), 1), (dict(cache_dtype=4, k_scale=66), 1),
]


@pytest.mark.parametrize("change,code", CACHE_REFUSALS + [
    (dict(T=-1), 1), (dict(hq=0), 1), (dict(rot=-2), 1), (dict(rot=130), 1), (dict(rot=31), 1), (dict(rot=40), 2),
    (dict(rot=31, interleaved=1), 1), (dict(dtype=3), 2), (dict(eps=-1.0), 1), (dict(qn=256), 1), (dict(kn=256), 1),
    (dict(ws=0), 3), (dict(ws_bytes=255), 3), (dict(ws=4112), 3), (dict(q=0), 1), (dict(q_out=0), 1), (dict(slots=0), 1),
    (dict(positions=0), 1), (dict(inv_freq=0), 1), (dict(q=258), 1), (dict(qn=258, kn=256), 1), (dict(slots=4100), 1),
    (dict(qt=1020), 2), (dict(oh=124), 2), (dict(hq=1 << 21), 2),
])
def test_rope_append_refusals(m, change, code):
    assert _rope(m, **change) == code, m.moe_last_error()
    assert m.moe_last_error() != ""


@pytest.mark.parametrize("change,code", CACHE_REFUSALS + [
    (dict(B=-1), 1), (dict(hq=0), 1), (dict(max_pages=-1), 1), (dict(window=-1), 1), (dict(hq=6), 1), (dict(dtype=3), 2),
    (dict(hq=1 << 17), 2), (dict(ws=0), 3), (dict(ws_bytes=4096), 3), (dict(ws=4112), 3), (dict(q=0), 1),
    (dict(out=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(q=258), 1), (dict(out=520), 1), (dict(lse=2), 1),
    (dict(qs=1020), 2), (dict(oh=124), 2),
])
def test_paged_attention_refusals(m, change, code):
    assert _attn(m, **change) == code, m.moe_last_error()
    assert m.moe_last_error() != ""


def test_without_tokens_or_sequences_nothing_runs(m):
    assert _rope(m, T=0, q=0, k=0, v=0, q_out=0, positions=0, slots=0, inv_freq=0) == 0
    assert _attn(m, B=0, q=0, out=0, table=0, lens=0) == 0
    lib, vp = m.library(), ctypes.c_void_p
    assert lib.moe_rope_append(None, m._ROPE_T.pack(*ROPE.values()), vp(4096), 1 << 26, None) == 1
    assert lib.moe_rope_append(m._CACHE_T.pack(*CACHE.values()), None, vp(4096), 1 << 26, None) == 1
    assert lib.moe_paged_attention(None, m._ATTN_T.pack(*ATTN.values()), vp(4096), 1 << 26, None) == 1
    assert lib.moe_paged_attention(m._CACHE_T.pack(*CACHE.values()), None, vp(4096), 1 << 26, None) == 1


def test_attention_workspace_bytes(m):
    lib = m.library()
    small = lib.moe_attention_workspace_bytes(m._CACHE_T.pack(*CACHE.values()), 8)
    # partial outputs of up to 320 CTAs, two each, 8 padded heads of 128
    assert small >= 640 * 8 * 128 * 4 and small % 256 == 0
    assert lib.moe_attention_workspace_bytes(m._CACHE_T.pack(*CACHE.values()), 64) >= 2 * 640 * 8 * 128 * 4
    assert lib.moe_attention_workspace_bytes(m._CACHE_T.pack(*CACHE.values()), 6) == 0
    assert lib.moe_attention_workspace_bytes(m._CACHE_T.pack(*{**CACHE, "head_dim": 512}.values()), 8) == 0


def test_packed_structs_have_the_headers_layout(m):
    """Sizes of the C structs (fields in declaration order, natural alignment,
    rounded up to 8 bytes)."""
    assert m._NORM_T.size == 6 * 8 + 4 * 8 + 6 * 4
    assert m._CACHE_T.size == 4 * 8 + 6 * 8 + 5 * 4 + 4
    assert m._ROPE_T.size == 9 * 8 + 8 * 8 + 6 * 4
    assert m._ATTN_T.size == 5 * 8 + 5 * 8 + 6 * 4
    assert struct.calcsize("@P") == 8


def test_binding_refuses_before_the_library(m):
    bf = torch.bfloat16
    x, w = torch.zeros(2, 64, dtype=bf), torch.zeros(64, dtype=bf)
    bad = [
        lambda: m.moe_add_rmsnorm(x, w, torch.zeros(2, 63, dtype=bf)),
        lambda: m.moe_add_rmsnorm(x, w, torch.zeros(2, 64, dtype=torch.float16)),
        lambda: m.moe_add_rmsnorm(x.float(), w, x),
        lambda: m.moe_add_rmsnorm(x[0], w, x[0]),
        lambda: m.moe_add_rmsnorm(x, w[:32], x),
        lambda: m.moe_add_rmsnorm(x, w, x, residual_out=x),
        lambda: m.moe_add_rmsnorm(x, w, x, scales=torch.zeros(2, 1)),
        lambda: m.moe_add_rmsnorm(x, w, x.to(torch.float8_e4m3fn)),
        lambda: m.moe_add_rmsnorm(x, w, x.to(torch.float8_e4m3fn), scales=torch.zeros(2, 2), group=64),
        lambda: m.moe_add_rmsnorm(x.t().contiguous().t(), w, x),
        lambda: m.moe_add_rmsnorm(x, w, x.clone()),  # not on a GPU
        lambda: m.MoeKvCache(torch.zeros(2, 16, 4), torch.zeros(2, 16, 4)),
        lambda: m.MoeKvCache(torch.zeros(2, 16, 1, 64), torch.zeros(2, 16, 1, 64)),
        lambda: m.MoeKvCache(torch.zeros(2, 16, 1, 64, dtype=bf), torch.zeros(2, 16, 2, 64, dtype=bf)),
        lambda: m.MoeKvCache(torch.zeros(2, 16, 1, 64, dtype=bf), torch.zeros(2, 16, 1, 64, dtype=bf), torch.ones(1)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    kv = torch.zeros(4, 16, 2, 64, dtype=bf)
    cache = m.MoeKvCache(kv, kv.clone())
    ws = m.alloc_attention_workspace(cache, 4)
    with pytest.raises(m.MoeError):
        m.alloc_attention_workspace(cache, 3)
    q, k = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 2, 64, dtype=bf)
    pos, f = torch.zeros(2, dtype=torch.int64), torch.zeros(32)
    table, lens = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q, ws),  # not on a GPU
        lambda: m.moe_rope_append(cache, q, k[:1], k, pos, pos, f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos.int(), pos, f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos[:1], f, q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f.double(), q, ws),
        lambda: m.moe_rope_append(cache, q, k, k, pos, pos, f, q, ws, q_norm_w=w),
        lambda: m.moe_rope_append(cache, q[:, :, :32], k, k, pos, pos, f, q, ws),
        lambda: m.moe_paged_attention(cache, q, table, lens, q.clone(), ws),  # not on a GPU
        lambda: m.moe_paged_attention(cache, q, table, lens.long(), q, ws),
        lambda: m.moe_paged_attention(cache, q, table[:1], lens, q, ws),
        lambda: m.moe_paged_attention(cache, q, table[0], lens, q, ws),
        lambda: m.moe_paged_attention(cache, q, table, lens, q.float(), ws),
        lambda: m.moe_paged_attention(cache, q, table, lens, q, ws, lse=torch.zeros(2, 3)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()

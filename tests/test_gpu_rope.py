"""moe_rope_append against its 64-bit form.  Errors before the rounding: the
angle to 2^-23 (a fraction of a turn in 24 bits), sine and cosine to 2^-22, the
per-head norm to 2^-19: under 2^-18 of the rotated pair's magnitudes."""
import pytest
import torch

from tests._layer_ref import E4M3_MAX, rope_ref, rounded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6
REL = 2.0 ** -18


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


def _run(m, T, hq, hkv, D, rot, page, dtype, e4m3=False, qk_norm=True, interleaved=False, head_major=False, far=0,
         joint=True, seed=0, base=10000.0, slots=None, in_place=False):
    g = torch.Generator().manual_seed(seed + T * 13 + D)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n_pages = -(-T // page) + 2
    qkv = rn(T, (hq + 2 * hkv) * D).to(dtype)
    cut = lambda t: (t[:, :hq * D].unflatten(1, (hq, D)), t[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D)),  # noqa: E731
                     t[:, (hq + hkv) * D:].unflatten(1, (hkv, D)))
    q, k, v = cut(qkv)
    pos = torch.arange(T) + far
    order = torch.randperm(n_pages, generator=g)
    t = torch.arange(T)
    if slots is None:
        slots = order[t // page] * page + t % page
    inv_freq = (base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1))).float()
    qn = (1 + 0.1 * rn(D)).to(dtype) if qk_norm else None
    kn = (1 + 0.1 * rn(D)).to(dtype) if qk_norm else None
    cdt = torch.float8_e4m3fn if e4m3 else dtype
    shape = (n_pages, hkv, page, D) if head_major else (n_pages, page, hkv, D)
    mark = 3.0
    kc, vc = (torch.full(shape, mark, device=DEV).to(cdt) for _ in range(2))
    if head_major:
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    ks = (0.01 + 0.02 * torch.rand(hkv, generator=g)) if e4m3 else None
    vs = (0.01 + 0.02 * torch.rand(hkv, generator=g)) if e4m3 else None
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    cache = m.MoeKvCache(kc, vc, dev(ks), dev(vs))
    ws = m.alloc_attention_workspace(cache, hq)
    if joint:
        qd, kd, vd = cut(qkv.to(DEV))
    else:  # heads outside the tokens
        qd, kd, vd = (u.to(DEV).transpose(0, 1).contiguous().transpose(0, 1) for u in (q, k, v))
    qo = qd if in_place else torch.empty(T, hq, D, dtype=dtype, device=DEV)
    m.moe_rope_append(cache, qd, kd, vd, pos.to(DEV), slots.to(DEV), inv_freq.to(DEV), qo, ws, q_norm_w=dev(qn),
                      k_norm_w=dev(kn), eps=EPS, interleaved=interleaved)
    ref, mag = rope_ref(q, qn, pos, inv_freq, EPS, interleaved)
    assert ((qo.cpu().double() - ref).abs() <= rounded(ref, dtype, 0.0, mag * REL)).all()
    kref, kmag = rope_ref(k, kn, pos, inv_freq, EPS, interleaved)
    got_k, got_v = kc.float().cpu().double(), vc.float().cpu().double()
    written = torch.zeros(n_pages, page, dtype=torch.bool)
    for i in range(T):
        s = int(slots[i])
        if s < 0 or s >= n_pages * page:
            continue
        p, o = s // page, s % page
        written[p, o] = True
        if e4m3:
            for got, ref, mg, sc in ((got_k[p, o], kref[i], kmag[i], ks), (got_v[p, o], v[i].double(), v[i].double().abs(), vs)):
                z = (ref / sc.double()[:, None])
                zc = z.clamp(-E4M3_MAX, E4M3_MAX)
                tol = torch.maximum(z.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) + 2 * REL * mg / sc.double()[:, None]
                assert ((got - zc).abs() <= tol).all()
        else:
            assert ((got_k[p, o] - kref[i]).abs() <= rounded(kref[i], dtype, 0.0, kmag[i] * REL)).all()
            assert torch.equal(got_v[p, o], v[i].double())
    kept = torch.full((1,), mark).to(cdt).double().item()
    assert (got_k[~written] == kept).all() and (got_v[~written] == kept).all()
    return ws


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,hq,hkv,D,rot,page", [
    (1, 16, 2, 256, 64, 16), (33, 16, 2, 256, 256, 16), (5, 24, 8, 128, 128, 32), (7, 12, 12, 64, 32, 7),
    (3, 1, 1, 16, 16, 1), (70, 1, 1, 64, 64, 24), (21, 4, 1, 80, 80, 16), (9, 6, 3, 96, 32, 5), (40, 5, 1, 128, 64, 64),
    (300, 3, 1, 192, 128, 16), (13, 2, 1, 256, 256, 16),
])
def test_halves(m, T, hq, hkv, D, rot, page, e4m3, dtype):
    m.moe_query_status(_run(m, T, hq, hkv, D, rot, page, dtype, e4m3))


@pytest.mark.parametrize("D,rot", [(64, 64), (8, 6), (128, 30), (256, 256), (40, 2), (64, 0)])
def test_interleaved_pairs_and_partial_widths(m, D, rot):
    _run(m, 11, 4, 2, D, rot, 16, torch.bfloat16, interleaved=True)
    _run(m, 11, 4, 2, D, rot, 16, torch.float16, interleaved=True, qk_norm=False)


@pytest.mark.parametrize("far", [4095, 131071, 1048575, 2 ** 31 - 64, -5000])
@pytest.mark.parametrize("base", [10000.0, 1e7])
def test_far_positions(m, far, base):
    _run(m, 17, 4, 2, 128, 128, 16, torch.float16, qk_norm=False, far=far, base=base)


def test_layouts_and_in_place(m):
    _run(m, 29, 8, 4, 128, 128, 16, torch.bfloat16, head_major=True)
    _run(m, 29, 8, 4, 128, 64, 16, torch.bfloat16, joint=False)
    _run(m, 29, 8, 4, 128, 128, 16, torch.bfloat16, e4m3=True, head_major=True, joint=False)
    _run(m, 29, 8, 4, 256, 64, 16, torch.bfloat16, in_place=True)


def test_padding_and_slots_past_the_cache(m):
    slots = torch.tensor([0, -1, 17, 40, -7, 3])
    m.moe_query_status(_run(m, 6, 4, 2, 64, 64, 16, torch.bfloat16, slots=slots))  # 3 pages of 16
    for bad in (48, 2 ** 33):
        slots = torch.tensor([0, bad, 17])
        ws = _run(m, 3, 4, 2, 64, 64, 16, torch.bfloat16, slots=slots)
        with pytest.raises(m.MoeError) as ei:
            m.moe_query_status(ws)
        assert ei.value.code == 6 and "slot" in str(ei.value) and "1" in str(ei.value)
        m.moe_query_status(ws)  # cleared


def test_e4m3_saturates(m):
    kv = torch.zeros(1, 4, 1, 64, dtype=torch.float8_e4m3fn, device=DEV)
    cache = m.MoeKvCache(kv, kv.clone(), torch.full((1,), 1e-3, device=DEV), torch.full((1,), 1e-3, device=DEV))
    ws = m.alloc_attention_workspace(cache, 1)
    one = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    m.moe_rope_append(cache, one, one, -one, zero, zero, torch.zeros(16, device=DEV), one.clone(), ws)
    assert (cache.k[0, 0].float() == 448).all() and (cache.v[0, 0].float() == -448).all()
    assert (cache.k[0, 1:].float() == 0).all()


def test_no_tokens(m):
    kv = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    cache = m.MoeKvCache(kv, kv.clone())
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    z = torch.empty(0, dtype=torch.int64, device=DEV)
    m.moe_rope_append(cache, e, e, e, z, z, torch.zeros(32, device=DEV), e, m.alloc_attention_workspace(cache, 1))

"""Measured cases of the decoder-layer operators around the MoE block: the RMS
norm with the residual's addition (16-bit or e4m3 output), the rotation and
append of new keys and values to a paged cache, and the attention of one new
token per sequence over that cache.

``run`` computes an operator either in its plain form (elementary torch
operations in fp32, rounded once at the end) or, with ``own`` set, through the
package's entry points.  ``exact`` states the same results in fp64.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96  # rows whose largest magnitude is below this are scaled by it
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases
def _norm(name, T, H, dtype, residual, out, group=0, pad=0):
    c = {"op": "norm", "T": T, "H": H, "dtype": dtype, "residual": residual, "out": out, "group": group, "pad": pad}
    return {"name": name, **c} if name else c


def _append(name, T, hq, hkv, D, rot, dtype, cache, page, qk_norm, interleaved=False, head_major=False, far=4096,
            padding=0):
    c = {"op": "append", "T": T, "hq": hq, "hkv": hkv, "D": D, "rot": rot, "dtype": dtype, "cache": cache,
         "page": page, "qk_norm": qk_norm, "interleaved": interleaved, "head_major": head_major, "far": far,
         "padding": padding}
    return {"name": name, **c} if name else c


def _attn(name, B, longest, skew, empty, hq, hkv, D, dtype, cache, page, window=0, head_major=False):
    c = {"op": "attn", "B": B, "longest": longest, "skew": skew, "empty": empty, "hq": hq, "hkv": hkv, "D": D,
         "dtype": dtype, "cache": cache, "page": page, "window": window, "head_major": head_major}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One decode token at the block's width: the norm before attention or before the MoE block.
        _norm("norm_token", 1, 2048, "bf16", True, "same"),
        # A ragged chunk of a prefill whose projections take e4m3 rows with one scale per token.
        _norm("norm_chunk_e4m3", 509, 2048, "bf16", True, "e4m3"),
        # A width that is no multiple of 8, in rows cut out of wider ones (a slice of a joint projection).
        _norm("norm_odd_slice", 1531, 1447, "fp16", False, "same", 0, 61),
        # A long prefill of a wide model with one scale per 128 columns: the largest norm.
        _norm("norm_prefill_groups", 16384, 4096, "bf16", True, "e4m3", 128),
        # One decode token: 16 query heads over 2 key/value heads of 256, a quarter of each rotated, per-head norms.
        _append("append_token", 1, 16, 2, 256, 64, "bf16", "bf16", 16, True),
        # A prefill chunk of the same heads: the largest append.
        _append("append_prefill", 8192, 16, 2, 256, 64, "bf16", "bf16", 16, True, far=131072),
        # An e4m3 cache with a scale per head, pages of 32 with the heads outside the tokens, padded tokens.
        _append("append_e4m3", 777, 24, 8, 128, 128, "fp16", "e4m3", 32, False, head_major=True, padding=37),
        # A decode batch of small heads, neighbouring pairs rotated, positions near a million.
        _append("append_pairs_far", 96, 12, 12, 64, 32, "bf16", "bf16", 24, False, interleaved=True, far=1048576),
        # One sequence in mid-conversation: the latency of one decode step's attention.
        _attn("attn_token", 1, 1531, 1.0, 0, 16, 2, 256, "bf16", "bf16", 16),
        # A serving batch of ragged lengths up to 32k tokens: the largest attention in 16 bits.
        _attn("attn_batch", 64, 32768, 1.0, 1, 16, 2, 256, "bf16", "bf16", 16),
        # One very long document beside two short requests, e4m3 cache, groups of 5 heads.
        _attn("attn_long_e4m3", 3, 262139, 6.0, 0, 40, 8, 128, "bf16", "e4m3", 64, head_major=True),
        # Many short sequences of ungrouped small heads with a sliding window, pages of 24 tokens.
        _attn("attn_window", 250, 3001, 1.0, 3, 12, 12, 64, "fp16", "fp16", 24, 512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "norm":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            H = max(8, H // 8 * 8)
        T = _log(rng, 1, max(1, min(16384, 67_000_000 // H)))
        out = rng.choice(["same", "same", "e4m3"])
        group = rng.choice([0, 64, 128]) if out == "e4m3" and H % 8 == 0 else 0
        pad = rng.choice([0, 0, 8, 64]) if H % 8 == 0 else rng.choice([0, 5])
        return _norm(None, T, H, dtype, rng.random() < 0.7, out, group, pad)
    D = rng.choice([64, 64, 96, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    cache = rng.choice([dtype, dtype, "e4m3"])
    page = rng.choice([1, 8, 16, 16, 20, 32, 64, 128])
    head_major = rng.random() < 0.5
    if kind == "append":
        rot = rng.choice([r for r in (32, 64, 96, 128, 256) if r <= D])
        T = _log(rng, 1, max(1, min(8192, 80_000_000 // ((hkv * G + 2 * hkv) * D * 2))))
        return _append(None, T, hkv * G, hkv, D, rot, dtype, cache, page, rng.random() < 0.5, rng.random() < 0.3,
                       head_major, rng.choice([4096, 131072, 1048576]), T // rng.choice([8, 100000]))
    B = _log(rng, 1, 256)
    # padded to the longest sequence the batch stays below the largest listed one
    cap = min(262144, 1_000_000_000 // (B * hkv * D))
    longest = _log(rng, 1, max(1, cap))
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    return _attn(None, B, longest, rng.choice([0.0, 0.5, 1.0, 4.0]), rng.choice([0, 0, B // 9]), hkv * G, hkv, D, dtype,
                 cache, page, window, head_major)


def _lens(case):
    """The multiset of sequence lengths of an attention case: the i-th of B is
    longest * ((i + 1) / B) ** skew, the first `empty` of them zero."""
    B = case["B"]
    lens = [max(1, round(case["longest"] * ((i + 1) / B) ** case["skew"])) for i in range(B)]
    return [0] * case["empty"] + lens[case["empty"]:]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16 if dtype == torch.bfloat16 else torch.float32)
    return t.mul_(scale).add_(shift).to(dtype)


def _cache(g, case, n_pages, fill):
    """K and V [pages, page, heads, D]; stored with the heads outside the
    tokens of a page where head_major is set.  e4m3 caches are filled in
    16-bit pieces."""
    P, h, D = case["page"], case["hkv"], case["D"]
    shape = (n_pages, h, P, D) if case["head_major"] else (n_pages, P, h, D)
    both = []
    for _ in range(2):
        t = torch.zeros(shape, device="cuda", dtype=DT[case["cache"]])
        if fill:
            flat, step = t.view(-1), 1 << 28
            for a in range(0, flat.numel(), step):
                n = min(step, flat.numel() - a)
                r = torch.randn(n, generator=g, device="cuda", dtype=torch.float16)
                if case["cache"] == "e4m3":
                    r.mul_(16.0)
                flat[a:a + n].copy_(r.to(t.dtype))
        both.append(t.permute(0, 2, 1, 3) if case["head_major"] else t)
    scales = [None, None]
    if case["cache"] == "e4m3":
        scales = [torch.rand(h, generator=g, device="cuda") * 0.05 + 0.04 for _ in range(2)]
    return both[0], both[1], scales[0], scales[1]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DT[case["dtype"]]
        # activations of a decoder: unit spread with a few loud columns
        col = 1.0 + 15.0 * (torch.rand(H, generator=g, device="cuda") < 0.01).float()
        x = _randn(g, T, H + case["pad"])
        x[:, :H].mul_(col)
        s["x"] = x.to(dt)[:, :H]
        s["weight"] = _randn(g, H, dtype=dt, scale=0.1, shift=1.0)
        s["residual"] = _randn(g, T, H, dtype=dt, scale=3.0) if case["residual"] else None
        s["residual_out"] = torch.empty(T, H, device="cuda", dtype=dt) if case["residual"] else None
        e4m3 = case["out"] == "e4m3"
        s["out_t"] = torch.empty(T, H, device="cuda", dtype=DT["e4m3"] if e4m3 else dt)
        n = -(-H // case["group"]) if case["group"] else 1
        s["scales"] = torch.empty(T, n, device="cuda") if e4m3 else None
        return s
    hq, hkv, D, dt = case["hq"], case["hkv"], case["D"], DT[case["dtype"]]
    host = random.Random(seed)
    if case["op"] == "append":
        T, P = case["T"], case["page"]
        n_pages = -(-T // P) + 3
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(g, case, n_pages, False)
        # one joint projection, cut into the three
        qkv = _randn(g, T, (hq + 2 * hkv) * D, dtype=dt)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["k"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        s["v"] = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        order = torch.randperm(n_pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = order[t // P] * P + t % P
        if case["padding"]:
            slots[torch.randperm(T, generator=g, device="cuda")[:case["padding"]]] = -1
        s["slots"] = slots
        s["positions"] = t + host.randrange(max(1, case["far"] - T))
        i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (1e7 ** (-2.0 * i / case["rot"])).float()
        s["q_norm_w"] = _randn(g, D, dtype=dt, scale=0.1, shift=1.0) if case["qk_norm"] else None
        s["k_norm_w"] = _randn(g, D, dtype=dt, scale=0.1, shift=1.0) if case["qk_norm"] else None
        s["q_out"] = torch.empty(T, hq, D, device="cuda", dtype=dt)
        return s
    B, P = case["B"], case["page"]
    lens = _lens(case)
    host.shuffle(lens)
    need = [-(-n // P) for n in lens]
    n_pages = sum(need) + 3
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(g, case, n_pages, True)
    width = max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(need, device="cuda")
    first = torch.cumsum(count, 0) - count
    at = torch.arange(width, device="cuda")
    used = at[None, :] < count[:, None]
    s["block_table"] = torch.where(used, order[(first[:, None] + at).clamp_(max=n_pages - 1)], -1).to(torch.int32)
    s["seq_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["q"] = _randn(g, B, hq, D, dtype=dt, scale=1.5)
    s["out_t"] = torch.empty(B, hq, D, device="cuda", dtype=dt)
    s["lse"] = torch.empty(B, hq, device="cuda")
    return s


# --------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _own_norm(s):
    import moe_decode_expert_gb300 as m
    m.moe_add_rmsnorm(s["x"], s["weight"], s["out_t"], residual=s["residual"], residual_out=s["residual_out"],
                      scales=s["scales"], group=s["group"], eps=EPS)
    return {"out": s["out_t"], "residual": s["residual_out"], "scales": s["scales"]}


def _own_handle(s):
    """The cache's handle and the workspace, made at a program's first call."""
    import moe_decode_expert_gb300 as m
    if "cache_t" not in s:
        s["cache_t"] = m.MoeKvCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        s["ws"] = m.alloc_attention_workspace(s["cache_t"], s["hq"])
    return m, s["cache_t"], s["ws"]


def _own_append(s):
    m, cache, ws = _own_handle(s)
    m.moe_rope_append(cache, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["q_out"], ws,
                      q_norm_w=s["q_norm_w"], k_norm_w=s["k_norm_w"], eps=EPS, interleaved=s["interleaved"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attn(s):
    m, cache, ws = _own_handle(s)
    m.moe_paged_attention(cache, s["q"], s["block_table"], s["seq_lens"], s["out_t"], ws, window=s["window"],
                          lse=s["lse"])
    return {"out": s["out_t"], "lse": s["lse"]}


def _plain_norm(s):
    h = s["x"].float()
    res = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        res = h.to(s["residual"].dtype)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    if s["scales"] is None:
        return {"out": y.to(s["x"].dtype), "residual": res, "scales": None}
    T, H = y.shape
    group = s["group"] or H
    n = -(-H // group)
    blocks = torch.nn.functional.pad(y, (0, n * group - H)).view(T, n, group)
    scale = blocks.abs().amax(2).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (blocks / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, n * group)[:, :H]
    return {"out": q.to(torch.float8_e4m3fn), "residual": res, "scales": scale}


def _rotate_plain(u, cos, sin, rot, interleaved):
    a, b = (u[..., 0:rot:2], u[..., 1:rot:2]) if interleaved else (u[..., :rot // 2], u[..., rot // 2:rot])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((lo, hi), -1).flatten(-2) if interleaved else torch.cat((lo, hi), -1)
    return torch.cat((turned, u[..., rot:]), -1)


def _plain_append(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["q_norm_w"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_norm_w"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_norm_w"].float()
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate_plain(q, cos, sin, s["rot"], s["interleaved"])
    k = _rotate_plain(k, cos, sin, s["rot"], s["interleaved"])
    kc, vc = s["k_cache"], s["v_cache"]
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    slots = s["slots"]
    # padded tokens rewrite what the first kept token writes, so nothing waits for a count
    kept = (slots >= 0).to(torch.int64).argmax()
    token = torch.where(slots >= 0, torch.arange(slots.numel(), device=slots.device), kept)
    at = slots[token]
    page, off = at // s["page"], at % s["page"]
    kc[page, off] = k.to(kc.dtype)[token]
    vc[page, off] = v.to(vc.dtype)[token]
    return {"q": q.to(s["q"].dtype), "k_cache": kc, "v_cache": vc}


def _plain_attn(s):
    B, hq, D = s["q"].shape
    hkv, P = s["hkv"], s["page"]
    table = s["block_table"].long().clamp(min=0)
    L = table.shape[1] * P
    k = s["k_cache"][table].reshape(B, L, hkv, D).float()
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    scores = torch.einsum("bhgd,blhd->bhgl", q, k) * (1.0 / math.sqrt(D))
    del k
    if s["k_scale"] is not None:
        scores = scores * s["k_scale"][:, None, None]
    at = torch.arange(L, device=q.device)
    n = s["seq_lens"].long()[:, None]
    seen = at < n
    if s["window"]:
        seen = seen & (at >= n - s["window"])
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][table].reshape(B, L, hkv, D).float()
    v = v * seen[:, :, None, None]
    o = torch.einsum("bhgl,blhd->bhgd", p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    if s["v_scale"] is not None:
        o = o * s["v_scale"][:, None, None]
    lse = torch.where(total > 0, top + torch.log(total), torch.full_like(total, -math.inf))
    return {"out": o.reshape(B, hq, D).to(s["q"].dtype), "lse": lse.reshape(B, hq)}


_run_own = {"norm": _own_norm, "append": _own_append, "attn": _own_attn}
_run_plain = {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn}


# ------------------------------------------------------------------- work
def work(case):
    sz = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n, e4m3 = case["T"] * case["H"], case["out"] == "e4m3"
        groups = -(-case["H"] // case["group"]) if case["group"] else 1
        b = n * sz * (3 if case["residual"] else 1) + n * (1 if e4m3 else sz) + case["H"] * sz
        return {"bytes": b + (case["T"] * groups * 4 if e4m3 else 0), "flops": n * (9 if e4m3 else 6)}
    hq, hkv, D = case["hq"], case["hkv"], case["D"]
    if case["op"] == "append":
        T, kept = case["T"], case["T"] - case["padding"]
        b = T * hq * D * sz * 2 + kept * 2 * hkv * D * (sz + SIZE[case["cache"]]) + T * 16 + case["rot"] * 2
        return {"bytes": b, "flops": T * (hq + hkv) * (3 * case["rot"] + (4 * D if case["qk_norm"] else 0))}
    tokens = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
    pages = sum(-(-n // case["page"]) for n in _lens(case))
    b = tokens * 2 * hkv * D * SIZE[case["cache"]] + case["B"] * hq * (2 * D * sz + 4) + pages * 4 + case["B"] * 4
    return {"bytes": b, "flops": 4 * tokens * hq * D}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """run()'s outputs from the operators' definitions in fp64, e4m3 values and
    16-bit values unrounded."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        rows = s["x"].to(f64)
        if s["residual"] is not None:
            rows += s["residual"].to(f64)
        ms = torch.einsum("th,th->t", rows, rows) / case["H"]
        y = torch.einsum("th,t,h->th", rows, 1.0 / torch.sqrt(ms + EPS), s["weight"].to(f64))
        scales = None
        if case["out"] == "e4m3":
            cols = case["group"] or case["H"]
            scales = torch.stack([part.abs().max(1).values for part in y.split(cols, 1)], 1)
            scales = torch.maximum(scales, torch.full_like(scales, AMAX_FLOOR)) / E4M3_MAX
            y = torch.cat([part / scales[:, i:i + 1] for i, part in enumerate(y.split(cols, 1))], 1)
        return {"out": y, "residual": rows if case["residual"] else None, "scales": scales}
    if case["op"] == "append":
        def norm(u, w):
            u = u.to(f64)
            return u if w is None else u / torch.sqrt((u * u).sum(2, keepdim=True) / case["D"] + EPS) * w.to(f64)

        turn = torch.outer(s["positions"].to(f64), s["inv_freq"].to(f64))
        z = torch.polar(torch.ones_like(turn), turn)[:, None, :]
        half = case["rot"] // 2

        def rotate(u):
            u = u.clone()
            i = torch.arange(half, device=u.device)
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            w = torch.complex(u[:, :, a], u[:, :, b]) * z
            u[:, :, a], u[:, :, b] = w.real, w.imag
            return u

        new = {"k": rotate(norm(s["k"], s["k_norm_w"])), "v": s["v"].to(f64)}
        out = {"q": rotate(norm(s["q"], s["q_norm_w"]))}
        kept = [(t, at) for t, at in enumerate(s["slots"].tolist()) if at >= 0]
        tok = torch.tensor([t for t, _ in kept], device="cuda", dtype=torch.int64)
        at = torch.tensor([a for _, a in kept], device="cuda", dtype=torch.int64)
        for n in ("k", "v"):
            c = s[n + "_cache"].to(f64)
            u = new[n][tok]
            if s[n + "_scale"] is not None:
                u = (u / s[n + "_scale"].to(f64)[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            c[at // case["page"], at % case["page"]] = u
            out[n + "_cache"] = c
        return out
    B, hq, hkv, D, P = (case[n] for n in ("B", "hq", "hkv", "D", "page"))
    out = torch.zeros(B, hq, D, device="cuda", dtype=f64)
    lse = torch.full((B, hq), -math.inf, device="cuda", dtype=f64)
    one = torch.ones(hkv, device="cuda", dtype=f64)
    ks = one if s["k_scale"] is None else s["k_scale"].to(f64)
    vs = one if s["v_scale"] is None else s["v_scale"].to(f64)
    for b, n in enumerate(s["seq_lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n <= lo:
            continue
        pos = torch.arange(lo, n, device="cuda")
        page, off = s["block_table"][b].long()[pos // P], pos % P
        for h in range(hkv):
            k = s["k_cache"][page, off, h].to(f64) * ks[h]
            v = s["v_cache"][page, off, h].to(f64) * vs[h]
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            z = s["q"][b, heads].to(f64) @ k.T / math.sqrt(D)
            total = torch.logsumexp(z, 1)
            lse[b, heads] = total
            out[b, heads] = torch.exp(z - total[:, None]) @ v
    return {"out": out, "lse": lse}

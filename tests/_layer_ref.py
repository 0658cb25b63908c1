"""Plain 64-bit forms of the layer operators (norm, rotation + append, paged
attention) on CPU tensors, and the error bounds their fp32 kernels are held to."""
import math

import torch

F64 = torch.float64
E4M3_MAX = 448.0


def half_step(dtype):
    """Largest relative rounding error of a type (normal values)."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Largest absolute rounding error among a type's subnormals."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def rounded(ref, dtype, rel=0.0, absolute=0.0):
    """Bound on |got - ref| for a result that is off by rel * |ref| + absolute
    before its one rounding to dtype."""
    h = half_step(dtype)
    return ref.abs() * (h + rel * (1 + h)) + absolute * (1 + h) + tiny(dtype)


def norm_ref(x, weight, residual, eps):
    h = x.to(F64) + (residual.to(F64) if residual is not None else 0.0)
    return h * torch.rsqrt((h * h).mean(1, keepdim=True) + eps) * weight.to(F64)


def scales_ref(y, group):
    H = y.shape[1]
    g = group or H
    s = torch.stack([p.abs().amax(1) for p in y.split(g, 1)], 1).clamp(min=2.0 ** -96) / E4M3_MAX
    return s, s.repeat_interleave(g, 1)[:, :H]


def rope_ref(u, norm_w, positions, inv_freq, eps, interleaved):
    """(rotated, the magnitude its rounding errors scale with)"""
    u = u.to(F64)
    if norm_w is not None:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + eps) * norm_w.to(F64)
    half = inv_freq.numel()
    a = positions.to(F64)[:, None, None] * inv_freq.to(F64)
    i = torch.arange(half)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out, mag = u.clone(), u.abs()
    out[..., p] = u[..., p] * a.cos() - u[..., q] * a.sin()
    out[..., q] = u[..., q] * a.cos() + u[..., p] * a.sin()
    both = u[..., p].abs() + u[..., q].abs()
    mag[..., p], mag[..., q] = both, both
    return out, mag


def gather(cache, table_row, tokens, page):
    t = torch.tensor(tokens, dtype=torch.int64)
    return cache[table_row.long()[t // page], t % page]


def attention_ref(q, k_cache, v_cache, table, lens, scale, window, k_scale, v_scale, weight_err):
    """out, lse and bounds on their errors before the output's rounding.
    weight_err: relative rounding error of a weight in the second product."""
    B, hq, D = q.shape
    n_pages, page, hkv, _ = k_cache.shape
    G = hq // hkv
    out = torch.zeros(B, hq, D, dtype=F64)
    err = torch.zeros(B, hq, D, dtype=F64)
    lse = torch.full((B, hq), -math.inf, dtype=F64)
    lse_err = torch.zeros(B, hq, dtype=F64)
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * page))
        lo = max(0, n - window) if window else 0
        tok = [j for j in range(lo, n) if 0 <= int(table[b, j // page]) < n_pages]
        if not tok:
            continue
        ks = gather(k_cache, table[b], tok, page).to(F64)
        vs = gather(v_cache, table[b], tok, page).to(F64)
        if k_scale is not None:
            ks = ks * k_scale.to(F64)[:, None]
            vs = vs * v_scale.to(F64)[:, None]
        for h in range(hq):
            k, v = ks[:, h // G], vs[:, h // G]
            qh = q[b, h].to(F64)
            s = scale * (k @ qh)
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, h])
            out[b, h] = p @ v
            # a score: D / 16 chained tensor steps, each off by at most a few
            # units of the last fp32 place of the sum of magnitudes; the shift
            # by the reference and the exponential add a little more
            ds = 2.0 ** -17 * abs(scale) * (k.abs() @ qh.abs()).max() + 2.0 ** -20
            # each chained step of the second product truncates by 2^-22 at most
            steps = len(tok) / 16 + 16
            w = 2 * ds + weight_err + steps * 2.0 ** -22
            err[b, h] = w * (p @ v.abs())
            lse_err[b, h] = ds + len(tok) * 2.0 ** -24 + 2.0 ** -22 * lse[b, h].abs() + 2.0 ** -20
    return out, lse, err, lse_err

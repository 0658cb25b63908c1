"""Plain 64-bit forms of the quantisation, the 8-bit product and the drawing of
tokens, on CPU tensors."""
import math

import torch

F64 = torch.float64
BLOCK = 128


def quant_ref(x, rows):
    """(x / scale unrounded, scales) of blocks of rows x 128."""
    x = x.to(F64)
    T, H = x.shape
    s = torch.stack([torch.stack([p.abs().max() for p in band.split(BLOCK, 1)]) for band in x.split(rows, 0)])
    s = torch.where(s < 2.0 ** -96, 2.0 ** -96, s) / 448.0
    return x / spread(s, rows, T, H), s


def spread(s, rows, T, H):
    return s.to(F64).repeat_interleave(rows, 0)[:T].repeat_interleave(BLOCK, 1)[:, :H]


def linear_ref(x, x_scales, w, w_scales):
    """(product, sum of the magnitudes of its terms)"""
    a = x.to(F64) * spread(x_scales, 1, *x.shape)
    b = w.to(F64) * spread(w_scales, BLOCK, *w.shape)
    return a @ b.t(), a.abs() @ b.abs().t()


def codes(T, K, g, pad=0, device="cpu"):
    """Random e4m3 rows in wider rows whose other bytes are NaN."""
    t = torch.full((T, K + pad), math.nan).to(torch.float8_e4m3fn)
    t[:, :K] = (torch.randn(T, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    return t.to(device)[:, :K]


def sample_ref(row, temperature, top_k, top_p, min_p, u):
    """(token, log-probability, how near the draw came to another token's border,
    relative to the whole sum) of one row."""
    row = row.to(F64)
    row = torch.where(row.isnan(), -math.inf, row)
    best = float(row.max())
    if best == -math.inf:
        return -1, -math.inf, 1.0
    order = sorted(range(len(row)), key=lambda i: (-float(row[i]), i)) if len(row) < 64 else \
        row.sort(dim=0, descending=True, stable=True)[1].tolist()
    temperature = 1.0 if math.isnan(temperature) else temperature
    if temperature <= 0 or min_p > 1 or top_p <= 0:
        order = order[:1]
    if top_k > 0:
        order = order[:top_k]
    at = torch.tensor(order)
    z = row[at]
    w = torch.where(z == best, 1.0, torch.exp((z - best) / max(temperature, 1e-30)))
    n, near = len(order), 1.0
    if top_p < 1 and n > 1:
        c = w.cumsum(0)
        n = 1 + int((c[:-1] < top_p * c[-1]).sum())
        near = min(near, float((c[:-1] - top_p * c[-1]).abs().min() / c[-1]))
    if min_p > 0:
        n = max(1, min(n, int((w >= min_p).sum())))
    at, back = at[:n].sort()
    w = w[:n][back]
    c = w.cumsum(0)
    u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0 ** -24)
    i = int((c <= u * c[-1]).sum())
    near = min(near, float((c - u * c[-1]).abs().min() / c[-1]))
    return int(at[i]), math.log(float(w[i] / c[-1])), near

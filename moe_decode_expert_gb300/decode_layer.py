"""Decoder layers around the MoE block, one new token per sequence and step.

A layer of the model the block belongs to is, for a batch of B sequences:

    y      = rmsnorm(x + r),  r = x + r             moe_add_rmsnorm
    q,k,v  = y Wqkv                                  a library product
    q, cache <- rotate(q), rotate(k), v              moe_rope_append
    a      = attention(q, cache)                     moe_paged_attention
    y      = rmsnorm(a Wo + r),  r = a Wo + r        moe_add_rmsnorm
    x      = moe(y)                                  moe_grouped_forward

x and r travel from layer to layer (the residual is added by the next norm).  A
step reads its positions, lengths and cache slots from device tensors that it
advances itself, so one captured graph serves every step.

    python -m moe_decode_expert_gb300.decode_layer --batch 8 --context 4096 --layers 4

builds random layers (hidden 2048, 16 query heads over 2 key/value heads of 256,
a quarter of each rotated; 256 experts, top-8, I 512, shared expert), fills the
caches to the context length, and prints the time of a decode step.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from . import (MOE_BF16, MoeCfg, MoeKvCache, alloc_attention_workspace, alloc_workspace, moe_add_rmsnorm,
               moe_grouped_forward, moe_paged_attention, moe_query_status, moe_rope_append)


@dataclass(frozen=True)
class LayerCfg:
    moe: MoeCfg
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    rot_dim: int
    rope_base: float = 1e7
    eps: float = 1e-6
    page_size: int = 16
    cache_e4m3: bool = False
    window: int = 0


def random_layer(cfg: LayerCfg, device, generator=None) -> dict:
    """One layer's weights, random at the scale of trained ones."""
    m, dt = cfg.moe, cfg.moe.torch_dtype
    rn = lambda *s, scale=0.02: (torch.randn(*s, generator=generator, device=device) * scale).to(dt)  # noqa: E731
    H, D = m.hidden, cfg.head_dim
    w = {"norm1": 1 + rn(H, scale=0.1), "norm2": 1 + rn(H, scale=0.1), "q_norm": 1 + rn(D, scale=0.1),
         "k_norm": 1 + rn(D, scale=0.1), "qkv": rn((cfg.n_q_heads + 2 * cfg.n_kv_heads) * D, H),
         "o": rn(H, cfg.n_q_heads * D), "router_w": rn(m.n_experts, H, scale=H ** -0.5),
         "w13": rn(m.n_experts, 2 * m.inter, H), "w2": rn(m.n_experts, H, m.inter), "shared_w13": None,
         "shared_w2": None, "shared_gate_w": None}
    if m.shared_inter:
        w["shared_w13"], w["shared_w2"] = rn(2 * m.shared_inter, H), rn(H, m.shared_inter)
    if m.has_shared_gate:
        w["shared_gate_w"] = rn(H)
    return w


def places(positions, block_table, page_size):
    """Cache slots (int64) and lengths (int32) of the tokens at ``positions``.  Positions
    are device values that a captured step counts up, so what they are is found out on
    the device: one outside the table gets slot -1 (nothing is stored) and a length
    that the attention clamps and records, and ``Decoder.check`` raises."""
    # (each operation is a launch of its own in a step, so there are as few as there can be)
    pages = block_table.shape[1]
    column = positions // page_size
    inside = column.clamp(0, pages - 1)
    slots = torch.add(positions % page_size, block_table.gather(1, inside[:, None])[:, 0], alpha=page_size)
    slots.masked_fill_(column != inside, -1)
    lens = torch.empty_like(block_table[:, 0], memory_format=torch.contiguous_format)
    torch.add(positions.clamp(-2, pages * page_size), 1, out=lens)
    return slots, lens


class Decoder:
    """Layers, their paged caches and everything a step needs, for ``batch``
    sequences of up to ``max_len`` tokens (rounded up to whole pages).  A sequence
    stepped past them loses its further tokens and is reported by ``check``."""

    def __init__(self, cfg: LayerCfg, layers: list[dict], batch: int, max_len: int, device):
        if not layers or batch < 1 or max_len < 1:
            raise ValueError("a decoder needs layers, and batch and max_len of at least 1")
        self.cfg, self.layers, self.B = cfg, layers, batch
        m, dt = cfg.moe, cfg.moe.torch_dtype
        H, D, hq, hkv, P = m.hidden, cfg.head_dim, cfg.n_q_heads, cfg.n_kv_heads, cfg.page_size
        pages = -(-max_len // P)
        self.max_len = pages * P
        # one pool of pages; every layer's cache uses the same table
        self.block_table = torch.randperm(batch * pages, device=device).view(batch, pages).to(torch.int32)
        cdt = torch.float8_e4m3fn if cfg.cache_e4m3 else dt
        self.caches = []
        for _ in layers:
            k, v = (torch.zeros(batch * pages, P, hkv, D, device=device, dtype=cdt) for _ in range(2))
            s = torch.full((hkv,), 0.05, device=device) if cfg.cache_e4m3 else None
            self.caches.append(MoeKvCache(k, v, s, s))
        i = torch.arange(cfg.rot_dim // 2, device=device, dtype=torch.float64)
        self.inv_freq = (cfg.rope_base ** (-2.0 * i / max(cfg.rot_dim, 1))).float()
        self.positions = torch.zeros(batch, dtype=torch.int64, device=device)
        self.ws_attn = alloc_attention_workspace(self.caches[0], hq)
        self.ws_moe = alloc_workspace(m, batch, device)
        e = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        self.y, self.x, self.r = e(batch, H), e(batch, H), e(batch, H)
        self.q, self.attn = e(batch, hq, D), e(batch, hq, D)
        self.ids, self.weights = e(batch, m.top_k, dtype=torch.int32), e(batch, m.top_k, dtype=torch.float32)

    def project(self, w, x, residual):
        """The norm before attention and the joint projection."""
        moe_add_rmsnorm(x, w["norm1"], self.y, residual=residual, residual_out=residual, eps=self.cfg.eps)
        return torch.matmul(self.y, w["qkv"].t())

    def attend(self, w, cache, qkv, slots, lens):
        """Rotation, append and attention of the step's tokens."""
        c, B = self.cfg, self.B
        hq, hkv, D = c.n_q_heads, c.n_kv_heads, c.head_dim
        q = qkv[:, :hq * D].unflatten(1, (hq, D))
        k = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        v = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        moe_rope_append(cache, q, k, v, self.positions, slots, self.inv_freq, self.q, self.ws_attn,
                        q_norm_w=w["q_norm"], k_norm_w=w["k_norm"], eps=c.eps)
        moe_paged_attention(cache, self.q, self.block_table, lens, self.attn, self.ws_attn, window=c.window)
        return torch.matmul(self.attn.view(B, hq * D), w["o"].t())

    def step(self, h):
        """One token per sequence: ``h`` [B, hidden] its embeddings; returns the
        last layer's block output and the residual it is still to be added to."""
        c = self.cfg
        slots, lens = places(self.positions, self.block_table, c.page_size)
        x = h
        for i, (w, cache) in enumerate(zip(self.layers, self.caches)):
            if i == 0:
                self.r.copy_(h)
                qkv = self.project(w, h, None)
            else:
                qkv = self.project(w, x, self.r)
            a = self.attend(w, cache, qkv, slots, lens)
            moe_add_rmsnorm(a, w["norm2"], self.y, residual=self.r, residual_out=self.r, eps=c.eps)
            moe_grouped_forward(c.moe, self.y, w["router_w"], w["w13"], w["w2"], w["shared_w13"], w["shared_w2"],
                                w["shared_gate_w"], self.ids, self.weights, self.x, self.ws_moe)
            x = self.x
        self.positions += 1
        return x, self.r

    def check(self):
        """Raises if a kernel recorded a device-side error."""
        moe_query_status(self.ws_attn)
        moe_query_status(self.ws_moe)


def full_width(**kw) -> LayerCfg:
    """The layer around the full-width block of the benchmark."""
    return LayerCfg(MoeCfg(2048, 256, 8, 512, 512, MOE_BF16, has_shared_gate=1), 16, 2, 256, 64, **kw)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=1)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--cache", choices=["same", "e4m3"], default="same")
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    cfg = full_width(cache_e4m3=a.cache == "e4m3")
    layers = [random_layer(cfg, dev) for _ in range(a.layers)]
    d = Decoder(cfg, layers, a.batch, a.context + a.steps + 16, dev)
    for cache in d.caches:  # a context as if it had been decoded
        for t in (cache.k, cache.v):
            t.copy_(torch.randn(t.shape, device=dev, dtype=torch.bfloat16) * (10 if a.cache == "e4m3" else 1))
    d.positions.fill_(a.context)
    h = torch.randn(a.batch, cfg.moe.hidden, device=dev).to(cfg.moe.torch_dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            d.step(h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.step(h)
    for _ in range(5):
        graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    n = max(1, a.steps - 8)
    begin.record()
    for _ in range(n):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    d.check()
    us = begin.elapsed_time(end) / n * 1e3
    print(f"batch {a.batch}, context {a.context}, {a.layers} layers, cache {a.cache}: "
          f"{us:.1f} us per step, {us / a.layers:.1f} us per layer")


if __name__ == "__main__":
    main()

"""Decoder layers around the MoE block, one new token per sequence and step.

A layer of the model the block belongs to is, for a batch of B sequences:

    y      = rmsnorm(x + r),  r = x + r             moe_add_rmsnorm
    q,k,v  = y Wqkv                                  a library product
    q, cache <- rotate(q), rotate(k), v              moe_rope_append
    a      = attention(q, cache)                     moe_paged_attention
    y      = rmsnorm(a Wo + r),  r = a Wo + r        moe_add_rmsnorm
    x      = moe(y)                                  moe_grouped_forward

x and r travel from layer to layer (the residual is added by the next norm).  With
``linear_e4m3`` the norm before attention writes e4m3 rows with a scale per 128
columns, attention's output is quantised alike (moe_quantize_e4m3), and both
products are moe_linear_e4m3 with weights quantised by blocks of 128 x 128.  With a
``head`` (random_head) a step begins and ends at tokens: the embedding's rows, and
after the layers a norm, the vocabulary's product (moe_linear_e4m3) and moe_sample.

A step reads its positions, lengths and cache slots from device tensors that it
advances itself, so one captured graph serves every step.

    python -m moe_decode_expert_gb300.decode_layer --batch 8 --context 4096 --layers 4

builds random layers (hidden 2048, 16 query heads over 2 key/value heads of 256,
a quarter of each rotated; 256 experts, top-8, I 512, shared expert), fills the
caches to the context length, and prints the time of a decode step; with
``--projections e4m3`` by 8-bit projections, with ``--vocab 151936`` from token to
token.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

from . import (MOE_BF16, MoeCfg, MoeKvCache, alloc_attention_workspace, alloc_status_workspace, alloc_workspace,
               moe_add_rmsnorm, moe_grouped_forward, moe_linear_e4m3, moe_paged_attention, moe_quantize_e4m3,
               moe_query_status, moe_rope_append, moe_sample)


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
    linear_e4m3: bool = False


def quantized(w):
    """A weight [N, K] as moe_linear_e4m3 takes it: e4m3 codes in rows of a multiple of
    16, and the scales of its 128 x 128 blocks."""
    N, K = w.shape
    q = torch.empty(N, -(-K // 16) * 16, dtype=torch.float8_e4m3fn, device=w.device)[:, :K]
    s = torch.empty(-(-N // 128), -(-K // 128), device=w.device)
    moe_quantize_e4m3(w, q, s, rows=128)
    return q, s


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
    if cfg.linear_e4m3:
        w["qkv"], w["o"] = quantized(w["qkv"]), quantized(w["o"])
    return w


def random_head(cfg: LayerCfg, vocab: int, device, generator=None) -> dict:
    """An embedding and a head for ``vocab`` tokens: the final norm's weight and the
    vocabulary's product, quantised."""
    H, dt = cfg.moe.hidden, cfg.moe.torch_dtype
    rn = lambda *s, scale: (torch.randn(*s, generator=generator, device=device) * scale).to(dt)  # noqa: E731
    return {"embed": rn(vocab, H, scale=1.0), "norm": 1 + rn(H, scale=0.1), "out": quantized(rn(vocab, H, scale=H ** -0.5))}


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

    def __init__(self, cfg: LayerCfg, layers: list[dict], batch: int, max_len: int, device, head: dict | None = None):
        if not layers or batch < 1 or max_len < 1:
            raise ValueError("a decoder needs layers, and batch and max_len of at least 1")
        if (cfg.linear_e4m3 or head is not None) and cfg.moe.hidden % 16:
            raise ValueError("8-bit products need a hidden size of a multiple of 16")
        if cfg.linear_e4m3 and cfg.n_q_heads * cfg.head_dim % 16:
            raise ValueError("8-bit products need query heads of a multiple of 16 values in all")
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
        self.head = head
        if cfg.linear_e4m3 or head is not None:
            f8, f32 = torch.float8_e4m3fn, torch.float32
            self.ws_linear = alloc_status_workspace(device)
            self.y8, self.y8_s = e(batch, H, dtype=f8), e(batch, -(-H // 128), dtype=f32)
            self.a8, self.a8_s = e(batch, hq * D, dtype=f8), e(batch, -(-hq * D // 128), dtype=f32)
            self.qkv, self.a = e(batch, (hq + 2 * hkv) * D), e(batch, H)
        if head is not None:
            self.tokens = torch.zeros(batch, dtype=torch.int64, device=device)
            self.h, self.logits = e(batch, H), e(batch, head["out"][0].shape[0], dtype=torch.float32)
            self.logprobs = e(batch, dtype=torch.float32)

    def norm_e4m3(self, x, weight, residual):
        moe_add_rmsnorm(x, weight, self.y8, residual=residual, residual_out=residual, scales=self.y8_s, group=128,
                        eps=self.cfg.eps)

    def project(self, w, x, residual):
        """The norm before attention and the joint projection."""
        if self.cfg.linear_e4m3:
            self.norm_e4m3(x, w["norm1"], residual)
            moe_linear_e4m3(self.y8, self.y8_s, *w["qkv"], self.qkv, self.ws_linear)
            return self.qkv
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
        if c.linear_e4m3:
            moe_quantize_e4m3(self.attn.view(B, hq * D), self.a8, self.a8_s)
            moe_linear_e4m3(self.a8, self.a8_s, *w["o"], self.a, self.ws_linear)
            return self.a
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

    def next_tokens(self, uniforms, **asked):
        """One token per sequence: steps by the tokens in ``self.tokens`` (which it
        replaces by the drawn ones, and returns), drawn with ``uniforms`` [batch] by what
        ``asked`` gives of moe_sample's temperature, top_k, top_p and min_p."""
        if self.head is None:
            raise ValueError("a decoder without a head ends at the hidden state: use step")
        # (a row whose mask or values leave nothing has token -1, and goes on with token 0)
        torch.index_select(self.head["embed"], 0, self.tokens.clamp(min=0), out=self.h)
        x, r = self.step(self.h)
        self.norm_e4m3(x, self.head["norm"], r)
        moe_linear_e4m3(self.y8, self.y8_s, *self.head["out"], self.logits, self.ws_linear)
        moe_sample(self.logits, uniforms, self.tokens, logprobs=self.logprobs, **asked)
        return self.tokens

    def check(self):
        """Raises if a kernel recorded a device-side error."""
        moe_query_status(self.ws_attn)
        moe_query_status(self.ws_moe)
        if self.cfg.linear_e4m3 or self.head is not None:
            moe_query_status(self.ws_linear)


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
    ap.add_argument("--projections", choices=["same", "e4m3"], default="same")
    ap.add_argument("--vocab", type=int, default=0, help="tokens of a head (0: steps end at the hidden state)")
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    cfg = full_width(cache_e4m3=a.cache == "e4m3", linear_e4m3=a.projections == "e4m3")
    layers = [random_layer(cfg, dev) for _ in range(a.layers)]
    head = random_head(cfg, a.vocab, dev) if a.vocab else None
    d = Decoder(cfg, layers, a.batch, a.context + a.steps + 16, dev, head)
    for cache in d.caches:  # a context as if it had been decoded
        for t in (cache.k, cache.v):
            t.copy_(torch.randn(t.shape, device=dev, dtype=torch.bfloat16) * (10 if a.cache == "e4m3" else 1))
    d.positions.fill_(a.context)
    h = torch.randn(a.batch, cfg.moe.hidden, device=dev).to(cfg.moe.torch_dtype)
    full = lambda v: torch.full((a.batch,), v, device=dev)  # noqa: E731
    uniforms, asked = torch.rand(a.batch, device=dev), dict(temperature=full(0.7), top_k=full(20), top_p=full(0.8))
    asked["top_k"] = asked["top_k"].int()

    def step():
        if head is None:
            d.step(h)
        else:
            d.next_tokens(uniforms, **asked)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
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
    more = f", projections {a.projections}, vocabulary {a.vocab}" if a.vocab or a.projections != "same" else ""
    print(f"batch {a.batch}, context {a.context}, {a.layers} layers, cache {a.cache}{more}: "
          f"{us:.1f} us per step, {us / a.layers:.1f} us per layer")


if __name__ == "__main__":
    main()

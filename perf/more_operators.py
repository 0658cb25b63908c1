"""Measured cases of the 8-bit projections and the end of a decode step: rows and
weights quantised to e4m3 with fp32 scales of blocks of 128, the product of two
such matrices, and the drawing of a token from each row of logits (temperature,
top-k, top-p, min-p, one given random number per row).

``run`` computes an operator either in its plain form (elementary torch
operations, 32 bits; 64 where the draw compares sums with a border) or, with
``own`` set, through the package's entry points.  ``exact`` states the same
results in fp64.
"""
import math
import random

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96  # blocks whose largest magnitude is below this are scaled by it
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
# rows of a serving batch ask for different things: temperature, top_k, top_p, min_p
# (temperature 0: the largest logit; top_k 0, top_p 1 and min_p 0 ask for nothing)
KINDS = {
    "greedy": (0.0, 0, 1.0, 0.0),
    "whole": (1.0, 0, 1.0, 0.0),
    "few": (0.7, 20, 0.8, 0.0),
    "many": (1.0, 1000, 1.0, 0.0),
    "nucleus": (0.9, 0, 0.95, 0.0),
    "wide": (2.5, 0, 0.95, 0.0),
    "minp": (1.5, 0, 1.0, 0.05),
    "all": (0.8, 200, 0.9, 0.02),
}


# ------------------------------------------------------------------- cases
def _quant(name, T, H, dtype, rows=1, pad=0):
    c = {"op": "quant", "T": T, "H": H, "dtype": dtype, "rows": rows, "pad": pad}
    return {"name": name, **c} if name else c


def _linear(name, M, N, K, out, pad=0):
    c = {"op": "linear", "M": M, "N": N, "K": K, "out": out, "pad": pad}
    return {"name": name, **c} if name else c


def _sample(name, B, V, dtype, kinds, spread=2.5, masked=0.0, empty=0, pad=0):
    c = {"op": "sample", "B": B, "V": V, "dtype": dtype, "kinds": kinds, "spread": spread, "masked": masked,
         "empty": empty, "pad": pad}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One decode token's attention output (16 heads of 256) before the output projection.
        _quant("quant_token", 1, 4096, "bf16"),
        # The same rows of a prefill chunk: the largest quantisation of activations.
        _quant("quant_prefill", 8192, 4096, "bf16"),
        # A weight of a ragged width as it is loaded, one scale per 128 x 128 block, cut out of wider rows.
        _quant("quant_weight", 5120, 2003, "fp16", 128, 5),
        # One decode token's joint query, key and value projection (16 + 2 * 2 heads of 256, hidden 2048).
        _linear("linear_token", 1, 5120, 2048, "bf16"),
        # The output projection of a decode batch.
        _linear("linear_batch", 48, 2048, 4096, "bf16"),
        # The vocabulary's logits of a small decode batch: the largest weight.
        _linear("linear_head", 8, 151936, 2048, "fp32"),
        # A ragged chunk through a product whose sizes are no multiples of the blocks.
        _linear("linear_chunk", 777, 1447, 2000, "fp16", 16),
        # A prefill chunk through the joint projection of a wider model: the largest product.
        _linear("linear_prefill", 8192, 5120, 4096, "bf16"),
        # One conversation's next token from the whole vocabulary: latency.
        _sample("sample_token", 1, 151936, "fp32", "few"),
        # A serving batch in which every request asks for something else.
        _sample("sample_batch", 64, 151936, "bf16", "mixed"),
        # Flat distributions of which 95 % are kept: the largest drawing.
        _sample("sample_flat", 256, 131072, "fp32", "wide"),
        # A small vocabulary of which a grammar allows few tokens, in some rows none.
        _sample("sample_masked", 33, 1003, "fp16", "mixed", masked=0.9, empty=2, pad=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quant", "linear", "linear", "sample", "sample"])
    if kind == "quant":
        H = _log(rng, 16, 16384)
        if rng.random() < 0.7:
            H = H // 8 * 8
        T = _log(rng, 1, min(16384, 33_000_000 // H))
        return _quant(None, T, H, rng.choice(["bf16", "fp16"]), rng.choice([1, 1, 128]), rng.choice([0, 0, 8, 3]))
    if kind == "linear":
        K = max(16, _log(rng, 16, 8192))
        pad = (-K) % 16 + rng.choice([0, 0, 16, 64])
        M = _log(rng, 1, 8192)
        most = min(151936, 300_000_000 // K, 170_000_000_000 // (M * K), 500_000_000 // M)
        N = _log(rng, min(16, most), most)
        return _linear(None, M, N, K, rng.choice(["bf16", "fp16", "fp32"]), pad)
    V = _log(rng, 32, 262144)
    B = _log(rng, 1, min(512, 33_000_000 // V))
    masked = rng.choice([0.0, 0.0, 0.0, 0.5, 0.99])
    return _sample(None, B, V, rng.choice(["bf16", "fp16", "fp32"]), rng.choice(["mixed", "mixed", *KINDS]),
                   rng.choice([0.3, 1.0, 2.5, 4.0]), masked, B // 8 if masked else 0, rng.choice([0, 0, 1, 64]))


# ------------------------------------------------------------------ inputs
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _codes(g, rows, cols, pad):
    """An e4m3 matrix of quantised normal values, in rows of cols + pad, filled in pieces."""
    t = torch.zeros(rows, cols + pad, device="cuda", dtype=torch.float8_e4m3fn)
    step = max(1, (1 << 27) // (cols + pad))
    for a in range(0, rows, step):
        n = min(step, rows - a)
        r = _randn(g, n, cols, dtype=torch.bfloat16).mul_(448.0 / 3.5).clamp_(-448.0, 448.0)
        t[a:a + n, :cols] = r.to(t.dtype)
    return t[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quant":
        T, H = case["T"], case["H"]
        # unit spread with a few loud columns
        loud = 1.0 + 15.0 * (torch.rand(H, generator=g, device="cuda") < 0.01).float()
        x = _randn(g, T, H + case["pad"])
        x[:, :H].mul_(loud)
        s["x"] = x.to(DT[case["dtype"]])[:, :H]
        s["q"] = torch.empty(T, H, device="cuda", dtype=torch.float8_e4m3fn)
        s["scales"] = torch.empty(-(-T // case["rows"]), -(-H // BLOCK), device="cuda")
        return s
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        s["x"] = _codes(g, M, K, case["pad"])
        s["w"] = _codes(g, N, K, case["pad"])
        # scales as the quantisation leaves them: activations of unit spread, weights of 0.02
        s["x_scales"] = (0.75 + 0.5 * torch.rand(M, kb, generator=g, device="cuda")) * (3.5 / 448.0)
        s["w_scales"] = (0.75 + 0.5 * torch.rand(-(-N // BLOCK), kb, generator=g, device="cuda")) * (0.07 / 448.0)
        s["out_t"] = torch.empty(M, N, device="cuda", dtype=DT[case["out"]])
        return s
    B, V = case["B"], case["V"]
    host = random.Random(seed)
    logits = _randn(g, B, V + case["pad"]).mul_(case["spread"])
    # a few tokens that the context makes likely
    near = torch.randint(0, V, (B, 1), generator=g, device="cuda")
    near = (near + torch.arange(12, device="cuda") * max(1, V // 13)) % V
    logits.scatter_add_(1, near, torch.rand(B, 12, generator=g, device="cuda").mul_(5.0 * case["spread"]))
    if case["masked"]:
        logits[torch.rand(logits.shape, generator=g, device="cuda") < case["masked"]] = -math.inf
    if case["empty"]:
        logits[torch.randperm(B, generator=g, device="cuda")[:case["empty"]]] = -math.inf
    s["logits"] = logits.to(DT[case["dtype"]])[:, :V]
    names = list(KINDS) if case["kinds"] == "mixed" else [case["kinds"]]
    ask = [KINDS[host.choice(names)] for _ in range(B)]
    s["temperature"] = torch.tensor([a[0] for a in ask], device="cuda")
    s["top_k"] = torch.tensor([a[1] for a in ask], device="cuda", dtype=torch.int32)
    s["top_p"] = torch.tensor([a[2] for a in ask], device="cuda")
    s["min_p"] = torch.tensor([a[3] for a in ask], device="cuda")
    s["uniforms"] = torch.rand(B, generator=g, device="cuda")
    s["tokens"] = torch.empty(B, device="cuda", dtype=torch.int64)
    s["logprobs"] = torch.empty(B, device="cuda")
    return s


# --------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _own_quant(s):
    import moe_decode_expert_gb300 as m
    m.moe_quantize_e4m3(s["x"], s["q"], s["scales"], rows=s["rows"])
    return {"q": s["q"], "scales": s["scales"]}


def _own_linear(s):
    import moe_decode_expert_gb300 as m
    if "ws" not in s:  # a program keeps one for all its calls
        s["ws"] = m.alloc_status_workspace(s["x"].device)
    m.moe_linear_e4m3(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out_t"], s["ws"])
    return s["out_t"]


def _own_sample(s):
    import moe_decode_expert_gb300 as m
    m.moe_sample(s["logits"], s["uniforms"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                 top_p=s["top_p"], min_p=s["min_p"], logprobs=s["logprobs"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def _plain_quant(s):
    T, H, rows = s["T"], s["H"], s["rows"]
    tb, hb = -(-T // rows), -(-H // BLOCK)
    x = torch.nn.functional.pad(s["x"].float(), (0, hb * BLOCK - H, 0, tb * rows - T)).view(tb, rows, hb, BLOCK)
    scales = x.abs().amax((1, 3)).clamp(min=AMAX_FLOOR) / E4M3_MAX
    q = (x / scales[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(tb * rows, hb * BLOCK)[:T, :H]
    return {"q": q.to(torch.float8_e4m3fn), "scales": scales}


def _plain_linear(s):
    N, K = s["w"].shape
    x = s["x"].float() * s["x_scales"].repeat_interleave(BLOCK, 1)[:, :K]
    w = s["w"].float() * s["w_scales"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return torch.einsum("mk,nk->mn", x, w).to(s["out_t"].dtype)


def _plain_sample(s):
    V = s["V"]
    l = s["logits"].double()
    l = torch.where(l.isnan(), -math.inf, l)
    top = l.amax(1, keepdim=True)
    t = s["temperature"].double()[:, None]
    # equal to the largest, infinite or not: weight 1; at temperature 0 no other has any
    w = torch.where(l == top, 1.0, torch.where(t > 0, torch.exp((l - top) / t.clamp(min=1e-30)), 0.0))
    order = l.sort(dim=1, descending=True, stable=True)[1]
    w = w.gather(1, order)
    rank = torch.arange(V, device=l.device)
    k = s["top_k"].long()[:, None]
    w = torch.where((k <= 0) | (rank < k), w, 0.0)
    cum = w.cumsum(1)
    before = torch.nn.functional.pad(cum[:, :-1], (1, 0))
    p = s["top_p"].double()[:, None]
    keep = (p >= 1) | (before < p * cum[:, -1:])
    keep &= w >= s["min_p"].double()[:, None]
    keep |= rank == 0
    keep &= (t > 0) | (rank == 0)
    w = torch.zeros_like(w).scatter(1, order, torch.where(keep, w, 0.0))
    cum = w.cumsum(1)
    total = cum[:, -1:]
    token = (cum <= s["uniforms"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    logprob = torch.log(w.gather(1, token) / total)
    none = top == -math.inf
    return {"tokens": torch.where(none, -1, token)[:, 0], "logprobs": torch.where(none, -math.inf, logprob)[:, 0].float()}


_run_own = {"quant": _own_quant, "linear": _own_linear, "sample": _own_sample}
_run_plain = {"quant": _plain_quant, "linear": _plain_linear, "sample": _plain_sample}


# ------------------------------------------------------------------- work
def work(case):
    if case["op"] == "quant":
        n = case["T"] * case["H"]
        scales = -(-case["T"] // case["rows"]) * -(-case["H"] // BLOCK)
        return {"bytes": n * (SIZE[case["dtype"]] + 1) + 4 * scales, "flops": 3 * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        return {"bytes": (M + N) * K + 4 * kb * (M - (-N // BLOCK)) + M * N * SIZE[case["out"]],
                "flops": 2 * M * N * K}
    n = case["B"] * case["V"]
    return {"bytes": n * SIZE[case["dtype"]] + case["B"] * 32, "flops": 5 * n}


# ------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """run()'s outputs from the operators' definitions in fp64, 16-bit and e4m3
    values unrounded."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "quant":
        bands, scales = [], []
        for band in s["x"].to(f64).split(case["rows"] if case["rows"] > 1 else case["T"], 0):
            parts = band.split(BLOCK, 1)
            amax = [p.abs().max(1, keepdim=True).values if case["rows"] == 1 else p.abs().max().view(1, 1) for p in parts]
            one = [a.clamp(min=AMAX_FLOOR) / E4M3_MAX for a in amax]
            bands.append(torch.cat([p / c for p, c in zip(parts, one)], 1))
            scales.append(torch.cat(one, 1))
        return {"q": torch.cat(bands), "scales": torch.cat(scales)}
    if case["op"] == "linear":
        # a block of K at a time, each weighted by its two scales afterwards
        out = torch.zeros(case["M"], case["N"], device="cuda", dtype=f64)
        column = torch.arange(case["N"], device="cuda") // BLOCK
        for i, a in enumerate(range(0, case["K"], BLOCK)):
            part = s["x"][:, a:a + BLOCK].to(f64) @ s["w"][:, a:a + BLOCK].to(f64).T
            part *= s["x_scales"][:, i, None].to(f64)
            part *= s["w_scales"][column, i].to(f64)
            out += part
        return out
    tokens, logprobs = [], []
    for b in range(case["B"]):
        row = s["logits"][b].to(f64)
        row[row.isnan()] = -math.inf
        temperature, k, p, m = (float(s[n][b]) for n in ("temperature", "top_k", "top_p", "min_p"))
        ranked, index = row.sort(dim=0, descending=True, stable=True)
        best = float(ranked[0])
        if best == -math.inf:
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        if temperature <= 0:
            tokens.append(int(index[0]))
            logprobs.append(0.0)
            continue
        if k > 0:
            ranked, index = ranked[:int(k)], index[:int(k)]
        mass = torch.exp((ranked - best) / temperature)
        mass[ranked == best] = 1.0
        n = len(mass)
        if p < 1:
            sums = mass.cumsum(0)
            n = 1 + int((sums[:-1] < p * sums[-1]).sum())
        n = max(1, min(n, int((mass >= m).sum())))
        kept, at = index[:n].sort()
        mass = mass[:n][at]
        sums = mass.cumsum(0)
        i = min(n - 1, int(torch.searchsorted(sums, s["uniforms"][b].to(f64) * sums[-1], right=True)))
        tokens.append(int(kept[i]))
        logprobs.append(math.log(float(mass[i] / sums[-1])))
    return {"tokens": torch.tensor(tokens, device="cuda"), "logprobs": torch.tensor(logprobs, device="cuda", dtype=f64)}

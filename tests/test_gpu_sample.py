"""moe_sample against its 64-bit form.  Weights are off by 2^-28 relative and 2^-44
of the largest, so a draw or a top-p border nearer than 2^-26 of the whole sum to
another token's is not asked to agree (u is drawn again there, on the CPU, before
the kernel runs).  A log-probability is a few fp32 operations: 2^-21 of its value,
and 2^-28 * 2 from the weights."""
import math

import pytest
import torch

from tests._projection_ref import sample_ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16
OFF = (1.0, 0, 1.0, 0.0)


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


def _refs(logits, asks, g):
    """uniforms and references, uniforms away from the borders."""
    us, refs = [], []
    for b, ask in enumerate(asks):
        ask = tuple(v if i == 1 else float(torch.tensor(v)) for i, v in enumerate(ask))  # as fp32 has them
        for _ in range(50):
            u = float(torch.rand(1, generator=g))
            r = sample_ref(logits[b], *ask, u)
            if r[2] > 2.0 ** -26:
                break
        us.append(u)
        refs.append(r)
    return torch.tensor(us), refs


def _run(m, logits, asks, us, **kw):
    B = logits.shape[0]
    t, k, p, q = (torch.tensor([a[i] for a in asks], dtype=torch.int32 if i == 1 else F32, device=DEV) for i in range(4))
    tokens = torch.full((B,), -7, dtype=torch.int64, device=DEV)
    lp = torch.full((B,), math.nan, device=DEV)
    m.moe_sample(logits, us.to(DEV), tokens, temperature=t, top_k=k, top_p=p, min_p=q, logprobs=lp, **kw)
    return tokens.cpu(), lp.cpu()


def _same(got, refs):
    tokens, lp = got
    assert tokens.tolist() == [r[0] for r in refs]
    for a, r in zip(lp.tolist(), refs):
        assert a == r[1] or abs(a - r[1]) <= 2.0 ** -21 * abs(r[1]) + 2.0 ** -27, (a, r)


ASKS = [OFF, (0.0, 0, 1.0, 0.0), (0.7, 20, 0.8, 0.0), (1.0, 1, 1.0, 0.0), (1.0, 50, 1.0, 0.0), (0.9, 0, 0.95, 0.0),
        (2.5, 0, 0.9, 0.0), (1.5, 0, 1.0, 0.05), (0.8, 200, 0.9, 0.02), (0.01, 0, 1.0, 0.0), (100.0, 0, 0.5, 0.0),
        (1.0, 0, 1e-6, 0.0), (1.0, 0, 1.0, 1.0), (1e-4, 5, 0.9, 0.0), (1.0, 10 ** 9, 2.0, -1.0), (1.0, -5, 0.99, 1e-7)]


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 500, 1003, 4097, 40000, 151936])
def test_every_kind_of_row(m, V, dtype):
    g = torch.Generator().manual_seed(V)
    asks = ASKS if V < 10 ** 5 else ASKS[:9]
    logits = torch.randn(len(asks), V, generator=g) * 3
    logits[:, V // 2] += 6
    logits = logits.to(dtype)
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV), asks, us), refs)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [37, 3000, 70000])
def test_ties_rank_by_index(m, V, dtype):
    """Few distinct values, so that every border falls among equal ones; -0 equals 0."""
    g = torch.Generator().manual_seed(V)
    logits = torch.randint(-1, 3, (12, V), generator=g).to(dtype)
    logits[logits == 0] = torch.where(torch.rand((logits == 0).sum(), generator=g) < 0.5, 0.0, -0.0).to(dtype)
    logits[3] = 1.5
    logits[4] = -0.0
    asks = [(1.0, 7, 1.0, 0.0), (1.0, V // 2, 1.0, 0.0), (1.0, 0, 0.3, 0.0), (1.0, 0, 0.77, 0.0), (1.0, V // 3, 0.41, 0.0),
            (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.2), (3.0, V - 1, 0.93, 0.0), (1.0, 3, 0.2, 0.0), OFF,
            (0.5, 0, 0.999, 0.9), (1.0, V, 0.6, 0.0)]
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV), asks, us), refs)


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("V", [50, 9000])
def test_masked_infinite_and_nan_logits(m, V, dtype):
    g = torch.Generator().manual_seed(V)
    logits = (torch.randn(9, V, generator=g) * 2).to(dtype)
    logits[0] = -math.inf
    logits[1] = math.nan
    logits[2, torch.rand(V, generator=g) < 0.95] = -math.inf
    logits[2, 7] = 1.0
    logits[3, ::3] = math.nan
    logits[4, [3, 11, 40]] = math.inf
    logits[5, 20] = math.inf
    logits[6] = torch.finfo(dtype).min
    logits[7] = torch.finfo(dtype).min
    logits[7, 33] = torch.finfo(dtype).max
    logits[8, 1:] = -math.inf
    for ask in (OFF, (0.7, 2, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (1.0, 0, 1.0, 0.3), (0.0, 0, 1.0, 0.0)):
        us, refs = _refs(logits, [ask] * 9, g)
        _same(_run(m, logits.to(DEV), [ask] * 9, us), refs)


def test_parameters_out_of_range(m):
    g = torch.Generator().manual_seed(5)
    nan, inf = math.nan, math.inf
    asks = [(nan, 0, nan, nan), (-1.0, 0, 1.0, 0.0), (1.0, 0, -3.0, 0.0), (1.0, 0, 1.0, 7.0), (1e-38, 0, 1.0, 0.0),
            (3e38, 0, 1.0, 0.0), (1.0, 2 ** 31 - 1, 1.0, 0.0), (1.0, -2 ** 31, 0.5, 0.0)]
    logits = torch.randn(len(asks), 777, generator=g)
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV), asks, us), refs)
    rows = logits[:1].expand(5, -1).contiguous()
    us = torch.tensor([nan, -2.0, 0.0, 1.0, inf])
    refs = [sample_ref(logits[0], *OFF, min(max(0.0 if math.isnan(u) else u, 0.0), 1 - 2.0 ** -24)) for u in us.tolist()]
    _same(_run(m, rows.to(DEV), [OFF] * 5, us), refs)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides_and_offsets(m, dtype):
    g = torch.Generator().manual_seed(6)
    for V, pad, off in ((1000, 1, 0), (1000, 7, 3), (999, 24, 5), (33, 0, 0)):
        wide = torch.full((5, V + pad + off), 50.0)
        wide[:, off:off + V] = torch.randn(5, V, generator=g)
        wide = wide.to(dtype)
        view = wide[:, off:off + V]
        us, refs = _refs(view, [ASKS[2]] * 5, g)
        _same(_run(m, wide.to(DEV)[:, off:off + V], [ASKS[2]] * 5, us), refs)


def test_defaults_and_many_rows(m):
    g = torch.Generator().manual_seed(7)
    logits = torch.randn(700, 100, generator=g)
    us, refs = _refs(logits, [OFF] * 700, g)
    tokens = torch.empty(700, dtype=torch.int64, device=DEV)
    m.moe_sample(logits.to(DEV), us.to(DEV), tokens)
    assert tokens.tolist() == [r[0] for r in refs]
    m.moe_sample(logits[:0].to(DEV), us[:0].to(DEV), tokens[:0])


def test_a_rows_result_depends_on_no_other_row(m):
    g = torch.Generator().manual_seed(8)
    logits = (torch.randn(64, 20000, generator=g) * 2).to(DEV)
    us = torch.rand(64, generator=g)
    asks = (ASKS * 4)[:64]
    tokens, lp = _run(m, logits, asks, us)
    for b in (0, 5, 6, 13, 63):
        t1, l1 = _run(m, logits[b:b + 1], asks[b:b + 1], us[b:b + 1])
        assert t1[0] == tokens[b] and l1[0] == lp[b]


@pytest.mark.parametrize("dtype,V", [(F32, 30000), (BF, 60001), (F32, 2049), (FP, 50007)])
def test_many_long_rows(m, dtype, V):
    """More rows than SMs: a CTA per row, which does not hold a long one in shared memory."""
    g = torch.Generator().manual_seed(V)
    B = 180
    logits = torch.randn(B, V + 3, generator=g) * torch.linspace(0.05, 4.0, B)[:, None]
    logits[::7] = (logits[::7] * 4).round() / 4  # ties
    logits = logits.to(dtype)
    asks = (ASKS[:9] * 20)[:B]
    view = logits[:, 3:]
    us, refs = _refs(view, asks, g)
    _same(_run(m, logits.to(DEV)[:, 3:], asks, us), refs)


@pytest.mark.parametrize("spread", [1e-6, 0.01, 0.3])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_nearly_flat_rows(m, dtype, spread):
    """Every filter ends among thousands of tokens of almost the same weight."""
    g = torch.Generator().manual_seed(3)
    logits = (torch.randn(10, 90000, generator=g) * spread + 5).to(dtype)
    asks = [OFF, (1.0, 0, 0.9, 0.0), (1.0, 45000, 1.0, 0.0), (1.0, 45000, 0.5, 0.0), (0.3, 0, 0.1, 0.0), (1.0, 3000, 0.7, 0.5),
            (1.0, 0, 0.5, 0.999), (1.0, 600, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (9.0, 89999, 0.99999, 0.0)]
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV), asks, us), refs)


@pytest.mark.parametrize("spread", [0.005, 0.05, 0.5])
@pytest.mark.parametrize("V", [20000, 131072])
def test_both_borders_among_tokens_of_one_weight(m, V, spread):
    """top_k ends inside a crowd of tokens of nearly one weight, and top_p of what it leaves as well."""
    g = torch.Generator().manual_seed(V)
    asks = [(1.0, V // 2, 0.97, 0.0), (1.0, V // 2, 0.5, 0.0), (0.5, V // 5, 0.999, 0.0), (1.0, V - 9, 0.9, 0.5),
            (2.0, 5000, 0.7, 0.0), (1.0, 3 * V // 4, 0.01, 0.0)]
    logits = torch.randn(len(asks), V, generator=g) * spread
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV), asks, us), refs)


@pytest.mark.parametrize("dtype,copies", [(F32, 1), (BF, 7), (FP, 40)])
def test_the_longest_rows(m, dtype, copies):
    """Few rows over a cluster each, and so many that they are read from memory again."""
    g = torch.Generator().manual_seed(copies)
    asks = [OFF, (0.7, 20, 0.8, 0.0), (1.0, 0, 0.95, 0.0), (1.3, 90000, 0.9, 1e-4)]
    logits = (torch.randn(len(asks), 393216, generator=g) * 2).to(dtype)
    us, refs = _refs(logits, asks, g)
    _same(_run(m, logits.to(DEV).repeat(copies, 1), asks * copies, us.repeat(copies)), refs * copies)


def test_draws_follow_the_weights(m):
    """Every token of a small row as often as its weight says: uniforms on a grid."""
    n = 4096
    row = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5])
    p = torch.softmax(row.double(), 0)
    us = (torch.arange(n) + 0.5) / n
    tokens, _ = _run(m, row.expand(n, -1).contiguous().to(DEV), [OFF] * n, us)
    counts = torch.bincount(tokens, minlength=5)
    assert ((counts.double() - n * p).abs() <= 1.0).all()  # a border each side, less than one grid step


def test_stream_and_graph(m):
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(3, 5000, generator=g)
    asks = ASKS[2:5]
    us, refs = _refs(logits, asks, g)
    side = torch.cuda.Stream()
    d = logits.to(DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = _run(m, d, asks, us, stream=side)
    side.synchronize()
    ud, tokens = us.to(DEV), torch.empty(3, dtype=torch.int64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_sample(d, ud, tokens)
    l2 = torch.randn(3, 5000, generator=g)
    u2, refs2 = _refs(l2, [OFF] * 3, g)
    d.copy_(l2)
    ud.copy_(u2)
    graph.replay()
    assert tokens.tolist() == [r[0] for r in refs2]
    del got, refs

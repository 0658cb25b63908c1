"""moe_paged_attention against its 64-bit form, with error bounds counted from
the kernel's arithmetic (tests/_layer_ref.py): scores and sums in fp32, weights
rounded to two bf16 terms (2^-17) or one fp16 term (2^-11) in the second
product, one rounding of the output."""
import math

import pytest
import torch

from tests._layer_ref import attention_ref, rounded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_decode_expert_gb300 as mod
    return mod


class Case:
    def __init__(self, m, lens, hq, hkv, D, page, dtype=torch.bfloat16, e4m3=False, head_major=False, seed=0, q_scale=1.5,
                 max_pages=None, junk=float("nan")):
        g = torch.Generator().manual_seed(seed + D * 31 + hq)
        self.m, self.lens, self.dtype, self.e4m3 = m, lens, dtype, e4m3
        B = len(lens)
        need = [-(-max(0, n) // page) for n in lens]
        width = max_pages if max_pages is not None else max(1, max(need))
        need = [min(n, width) for n in need]
        n_pages = sum(need) + 2
        order = torch.randperm(n_pages, generator=g)
        self.table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        cdt = torch.float8_e4m3fn if e4m3 else dtype
        # unwritten slots hold junk: NaN by default
        self.k, self.v = (torch.full((n_pages, page, hkv, D), junk).to(cdt) for _ in range(2))
        for b, n in enumerate(lens):
            for p in range(need[b]):
                m_ = min(page, n - p * page)
                for c in (self.k, self.v):
                    c[int(self.table[b, p]), :m_] = (torch.randn(m_, hkv, D, generator=g) * (8 if e4m3 else 1)).to(cdt)
        self.ks = (0.08 + 0.08 * torch.rand(hkv, generator=g)) if e4m3 else None
        self.vs = (0.08 + 0.08 * torch.rand(hkv, generator=g)) if e4m3 else None
        self.q = (torch.randn(B, hq, D, generator=g) * q_scale).to(dtype)
        self.head_major = head_major
        self.ws = None

    def run(self, window=0, scale=None, q=None, out=None, stream=None, ws=None, lse=True):
        m = self.m
        kd, vd = self.k.to(DEV), self.v.to(DEV)
        if self.head_major:
            kd, vd = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (kd, vd))
        dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        cache = m.MoeKvCache(kd, vd, dev(self.ks), dev(self.vs))
        hq = self.q.shape[1]
        self.ws = ws if ws is not None else m.alloc_attention_workspace(cache, hq)
        qd = self.q.to(DEV) if q is None else q
        out = torch.full(self.q.shape, 7.0, dtype=self.dtype, device=DEV) if out is None else out
        lse_t = torch.full(self.q.shape[:2], 7.0, device=DEV) if lse else None
        m.moe_paged_attention(cache, qd, self.table.to(DEV), torch.tensor(self.lens, dtype=torch.int32).to(DEV), out,
                              self.ws, scale=scale, window=window, lse=lse_t, stream=stream)
        torch.cuda.synchronize()
        return out.cpu(), lse_t.cpu() if lse else None

    def check(self, window=0, scale=None, status=True, **kw):
        out, lse = self.run(window, scale, **kw)
        sc = self.q.shape[2] ** -0.5 if scale is None else scale
        werr = 2.0 ** -17 if self.dtype == torch.bfloat16 and not self.e4m3 else 2.0 ** -11
        ref, rlse, err, lerr = attention_ref(self.q, self.k.float() if self.e4m3 else self.k,
                                             self.v.float() if self.e4m3 else self.v, self.table, self.lens, sc, window,
                                             self.ks, self.vs, werr)
        d = (out.double() - ref).abs()
        assert (d <= rounded(ref, self.dtype, 0.0, err)).all(), (d.max(), d.argmax())
        if lse is not None:
            gone = torch.isinf(rlse)
            assert torch.equal(lse.double()[gone], rlse[gone])
            assert ((lse.double() - rlse).abs()[~gone] <= lerr[~gone]).all()
        if status:
            self.m.moe_query_status(self.ws)
        return out, lse


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (3, 3), (32, 2)])
def test_ragged_lengths(m, D, hq, hkv, e4m3, dtype):
    Case(m, [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 700], hq, hkv, D, 16, dtype, e4m3).check()


@pytest.mark.parametrize("D", [16, 80, 96, 192, 240])
@pytest.mark.parametrize("e4m3", [False, True])
def test_head_dims_between(m, D, e4m3):
    Case(m, [33, 0, 257], 10, 2, D, 16, torch.float16, e4m3).check()
    if not e4m3:
        Case(m, [33, 1, 257], 4, 2, D - 8, 16).check()


@pytest.mark.parametrize("page", [1, 3, 7, 16, 20, 32, 48, 64, 128, 1000])
@pytest.mark.parametrize("head_major", [False, True])
def test_page_sizes_and_orders(m, page, head_major):
    Case(m, [1, 50, 333], 8, 2, 128, page, head_major=head_major).check()
    Case(m, [70, 129], 12, 12, 64, page, torch.float16, head_major=head_major).check()
    Case(m, [70, 129], 8, 2, 64, page, e4m3=True, head_major=head_major).check()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (9, 1), (16, 1), (17, 1), (20, 1), (33, 1), (64, 1), (40, 8)])
def test_groups(m, hq, hkv):
    Case(m, [200, 31, 0], hq, hkv, 128, 16).check()
    Case(m, [200, 31], hq, hkv, 256, 16, torch.float16).check()
    Case(m, [200, 31], hq, hkv, 64, 16, e4m3=True).check()


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 511, 10000])
def test_windows(m, window):
    Case(m, [0, 1, 16, 40, 512, 1023], 8, 2, 128, 16).check(window)
    Case(m, [0, 1, 16, 40, 512, 1023], 4, 4, 64, 24, torch.float16).check(window)
    Case(m, [0, 1, 16, 40, 512, 1023], 4, 2, 256, 7, e4m3=True).check(window)


@pytest.mark.parametrize("lens", [[4097], [20000, 3], [1, 9000, 1, 0, 5000], [2600] * 9, list(range(0, 400))])
def test_long_and_many(m, lens):
    """Sequences cut over many CTAs, CTAs that hold many sequences, joins of
    more parts than one CTA joins at a time."""
    Case(m, lens, 8, 1, 64, 16).check()
    if sum(lens) < 30000:
        Case(m, lens, 4, 2, 128, 16, torch.float16).check()


def test_strided_queries_and_outputs(m):
    c = Case(m, [100, 37], 8, 2, 128, 16)
    wide = torch.full((2, 12, 256), 5.0, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 2:10, 64:192]
    q.copy_(c.q)
    out = torch.full((8, 2, 192), 5.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    c.check(q=q, out=out[:, :, :128])
    assert (out[:, :, 128:] == 5).all()


def test_scale_and_sharp_scores(m):
    Case(m, [300, 90], 8, 2, 128, 16, q_scale=20.0).check()  # nearly one-hot
    Case(m, [300, 90], 8, 2, 128, 16).check(scale=-0.3)
    Case(m, [300, 90], 8, 2, 128, 16).check(scale=0.0)
    Case(m, [300, 90], 8, 2, 128, 16, q_scale=1e-6).check()
    Case(m, [300, 90], 8, 2, 128, 16, e4m3=True, q_scale=1e-30).check()  # bf16 queries far below fp16's range
    Case(m, [300, 90], 8, 2, 128, 16, e4m3=True, q_scale=1e6).check(scale=1e-7)


def test_flat_tail_beside_one_large_weight(m):
    """A weight of 1 beside 8000 of about 1e-7 each: the tail's share is kept."""
    c = Case(m, [8001], 1, 1, 64, 16, torch.float16, junk=0.0)
    c.q.fill_(1.0)
    c.k.zero_()
    c.v.fill_(1.0)
    first = int(c.table[0, 0])
    c.k[first, 0] = 2.0  # score 16 above the others: e^-16 = 1.1e-7
    c.v[first, 0] = -1.0
    c.check(scale=0.125)


def test_no_lse(m):
    Case(m, [100, 37], 8, 2, 128, 16).check(lse=False)


def test_non_finite_tokens(m):
    for e4m3 in (False, True):
        c = Case(m, [100, 64, 30], 8, 2, 128, 16, e4m3=e4m3)
        clean, _ = c.run()
        c.k[int(c.table[0, 1]), 3, 0] = float("nan")
        out, _ = c.run()
        assert out[0, :4].isnan().all() and torch.equal(out[0, 4:], clean[0, 4:]) and torch.equal(out[1:], clean[1:])
        # outside the window the same token is never read
        win, _ = c.run(window=50)
        assert torch.isfinite(win).all()
        c.v[int(c.table[2, 0]), 3, 1, 7] = float("nan")
        out, _ = c.run()
        bad = out[2].isnan()
        assert bad[4:, 7].all() and int(bad.sum()) == 4
    c = Case(m, [40], 2, 1, 64, 16, torch.float16)
    c.k[int(c.table[0, 0]), 5] = float("inf")
    c.q.fill_(1.0)
    assert c.run()[0].isnan().all()
    c.q.fill_(-1.0)  # one score of -infinity among finite ones counts nothing
    out, lse = c.run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_bad_pages_are_dropped_and_recorded(m):
    for bad in (-1, -2 ** 31, 2 ** 31 - 1, 1000):
        c = Case(m, [100, 64], 8, 2, 128, 16)
        c.table[0, 2] = bad
        c.check(status=False)
        with pytest.raises(m.MoeError) as ei:
            m.moe_query_status(c.ws)
        assert ei.value.code == 6 and "page" in str(ei.value) and "0" in str(ei.value)
        m.moe_query_status(c.ws)
    c = Case(m, [20], 8, 2, 64, 16)
    c.table[0] = -5
    out, lse = c.run()
    assert (out == 0).all() and (lse == -math.inf).all()
    with pytest.raises(m.MoeError):
        m.moe_query_status(c.ws)


def test_bad_lengths_are_clamped_and_recorded(m):
    for lens in ([-1, 40], [40, 49], [40, 2 ** 31 - 1], [-2 ** 31, 48]):
        c = Case(m, lens, 4, 2, 64, 16, max_pages=3, junk=0.5)
        c.check(status=False)
        with pytest.raises(m.MoeError) as ei:
            m.moe_query_status(c.ws)
        assert ei.value.code == 6 and "length" in str(ei.value)


def test_results_repeat_and_workspaces_are_shared_by_shapes(m):
    """Bitwise equal over repetitions (joins do not depend on arrival), and one
    workspace serves calls of other shapes in between."""
    big = Case(m, [9000, 40, 3000], 16, 2, 256, 16)
    small = Case(m, [5, 900], 8, 2, 64, 16, torch.float16)
    first, lse = big.check()
    ws = big.ws
    for _ in range(5):
        small.check(ws=ws)
        again, lse2 = big.run(ws=ws)
        assert torch.equal(first, again) and torch.equal(lse, lse2)


def test_other_stream_and_graph(m):
    c = Case(m, [700, 33], 8, 2, 128, 16)
    want, _ = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = c.run(stream=side)
    assert torch.equal(want, got)
    kd, vd, qd, td = c.k.to(DEV), c.v.to(DEV), c.q.to(DEV), c.table.to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    cache = m.MoeKvCache(kd, vd)
    ws = m.alloc_attention_workspace(cache, 8)
    out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_paged_attention(cache, qd, td, lens, out, ws)
    graph.replay()
    assert torch.equal(out.cpu(), want)
    lens.copy_(torch.tensor([1, 20], dtype=torch.int32))  # the same graph serves other lengths
    graph.replay()
    c.lens = [1, 20]
    want, _ = c.run()
    assert torch.equal(out.cpu(), want)


def test_offsets_past_32_bits(m):
    """A cache whose last pages lie more than 2^32 elements from its start."""
    page, hkv, D = 64, 8, 256
    n_pages = (2 ** 32) // (page * hkv * D) + 8
    k = torch.zeros(n_pages, page, hkv, D, dtype=torch.float8_e4m3fn, device=DEV)
    v = torch.zeros_like(k)
    cache = m.MoeKvCache(k, v)
    ws = m.alloc_attention_workspace(cache, 8)
    g = torch.Generator().manual_seed(3)
    new = torch.randn(2, 8, D, generator=g).to(torch.bfloat16).to(DEV)
    slots = torch.tensor([n_pages * page - 1, (n_pages - 2) * page], device=DEV)
    pos = torch.zeros(2, dtype=torch.int64, device=DEV)
    m.moe_rope_append(cache, new, new, new, pos, slots, torch.zeros(16, device=DEV), torch.empty_like(new), ws)
    assert torch.equal(k[-1, -1].float(), new[0].float().to(torch.float8_e4m3fn).float())
    table = torch.tensor([[n_pages - 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([1], dtype=torch.int32, device=DEV)
    out = torch.empty(1, 8, D, dtype=torch.bfloat16, device=DEV)
    m.moe_paged_attention(cache, new[:1], table, lens, out, ws)
    assert torch.equal(out[0].float(), new[1].float().to(torch.float8_e4m3fn).float())
    m.moe_query_status(ws)


@pytest.mark.parametrize("D,lens", [(256, [30000, 1, 2, 3, 4, 5]), (64, [3, 70000, 1, 1, 1])])
def test_two_levels_of_joins(m, D, lens):
    """More parts of one sequence than one CTA joins at a time."""
    c = Case(m, lens, 4, 1, D, 16)
    first, _ = c.check()
    again, _ = c.run(ws=c.ws)
    assert torch.equal(first, again)


def test_a_line_long_enough_to_keep_some_back(m):
    """Over 256 units per CTA: the last ones are taken by whoever gets done first;
    results stay the same from run to run.  The reference is formed on the GPU."""
    lens = [62500, 70000, 55001, 61000, 65537]
    page, hkv, hq, D = 16, 4, 8, 256
    need = [-(-n // page) for n in lens]
    g = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.randn(sum(need), page, hkv, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    order = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    table = torch.full((5, max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = (torch.randn(5, hq, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    cache = m.MoeKvCache(k, v)
    ws = m.alloc_attention_workspace(cache, hq)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(3):
        out, lse = torch.empty_like(q), torch.empty(5, hq, device=DEV)
        m.moe_paged_attention(cache, q, table, n, out, ws, lse=lse)
        outs.append((out, lse))
    m.moe_query_status(ws)
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    for b, length in enumerate(lens):
        pos = torch.arange(length, device=DEV)
        pages, off = table[b].long()[pos // page], pos % page
        for h in range(hkv):
            kh, vh = k[pages, off, h].double(), v[pages, off, h].double()
            qh = q[b, 2 * h:2 * h + 2].double()
            s = qh @ kh.T * D ** -0.5
            total = torch.logsumexp(s, 1)
            p = torch.exp(s - total[:, None])
            ref = p @ vh
            ds = 2.0 ** -17 * D ** -0.5 * (qh.abs() @ kh.abs().T).amax(1, keepdim=True) + 2.0 ** -20
            err = (2 * ds + 2.0 ** -17 + (length / 16 + 16) * 2.0 ** -22) * (p @ vh.abs())
            d = (outs[0][0][b, 2 * h:2 * h + 2].double() - ref).abs()
            assert (d <= rounded(ref, torch.bfloat16, 0.0, err)).all()
            tol = ds[:, 0] + length * 2.0 ** -24 + 2.0 ** -22 * total.abs() + 2.0 ** -20
            assert ((outs[0][1][b, 2 * h:2 * h + 2].double() - total).abs() <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", [(9, 1), (16, 1), (17, 1), (33, 1), (64, 1), (72, 1), (40, 2)])
def test_wide_rows_with_their_heads_on_several_lines(m, hq, hkv, e4m3):
    """Groups of more than 8 heads of 256, up to 8 lines and past them."""
    c = Case(m, [2700, 31, 0, 517], hq, hkv, 256, 16, torch.float16, e4m3)
    first, _ = c.check()
    again, _ = c.run(ws=c.ws)
    assert torch.equal(first, again)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,hq,hkv", [(64, 24, 2), (128, 40, 4), (256, 12, 1), (256, 64, 4), (96, 8, 8)])
def test_short_segments_with_a_cta_each(m, D, hq, hkv, e4m3):
    lens = [76, 0, 1, 16, 17, 33, 64, 65, 100, 76, 5, 48, 49, 31, 32, 128, 90, 3]
    c = Case(m, lens, hq, hkv, D, 16, e4m3=e4m3)
    c.check()
    c.check(window=20)


def test_long_lines_side_by_side(m):
    """Over 256 units per CTA on each of two lines."""
    lens = [110000, 108001, 105003]
    page, hkv, G, D = 16, 2, 12, 256
    need = [-(-n // page) for n in lens]
    g = torch.Generator(device=DEV).manual_seed(6)
    k, v = (torch.randn(sum(need), page, hkv, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    order = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    table = torch.full((3, max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    q = (torch.randn(3, G * hkv, D, generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    cache = m.MoeKvCache(k, v)
    ws = m.alloc_attention_workspace(cache, G * hkv)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    outs = []
    for _ in range(3):
        out, lse = torch.empty_like(q), torch.empty(3, G * hkv, device=DEV)
        m.moe_paged_attention(cache, q, table, n, out, ws, lse=lse)
        outs.append((out, lse))
    m.moe_query_status(ws)
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    for b, length in enumerate(lens):
        pos = torch.arange(length, device=DEV)
        pages, off = table[b].long()[pos // page], pos % page
        for h in range(hkv):
            kh, vh = k[pages, off, h].double(), v[pages, off, h].double()
            mine = slice(G * h, G * h + G)
            qh = q[b, mine].double()
            s = qh @ kh.T * D ** -0.5
            total = torch.logsumexp(s, 1)
            p = torch.exp(s - total[:, None])
            ref = p @ vh
            ds = 2.0 ** -17 * D ** -0.5 * (qh.abs() @ kh.abs().T).amax(1, keepdim=True) + 2.0 ** -20
            err = (2 * ds + 2.0 ** -17 + (length / 16 + 16) * 2.0 ** -22) * (p @ vh.abs())
            d = (outs[0][0][b, mine].double() - ref).abs()
            assert (d <= rounded(ref, torch.bfloat16, 0.0, err)).all()
            tol = ds[:, 0] + length * 2.0 ** -24 + 2.0 ** -22 * total.abs() + 2.0 ** -20
            assert ((outs[0][1][b, mine].double() - total).abs() <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(20, 1), (64, 1), (34, 2), (144, 1)])
def test_groups_of_several_chunks_in_a_wide_table(m, D, hq, hkv, e4m3):
    """Chunks of 16 heads on lines side by side; a table wide enough that the
    sequences are not known to be short."""
    c = Case(m, [1200, 31, 0, 517, 64, 3], hq, hkv, D, 64, torch.float16, e4m3, max_pages=400)
    first, _ = c.check()
    again, _ = c.run(ws=c.ws)
    assert torch.equal(first, again)


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("D,hq,hkv", [(64, 12, 12), (96, 14, 7), (128, 40, 8), (128, 60, 6), (128, 120, 4), (256, 36, 3)])
def test_kv_heads_on_lines_side_by_side(m, D, hq, hkv, head_major):
    c = Case(m, [900, 31, 0, 517, 64, 3, 1, 200, 16, 77, 130], hq, hkv, D, 32, torch.float16, True,
             head_major=head_major, max_pages=500)
    first, _ = c.check()
    again, _ = c.run(ws=c.ws)
    assert torch.equal(first, again)

"""Paged attention by single CTAs: what test_gpu_attention.py asks of a few sequences,
which teams of CTAs serve, asked again with further sequences beside them, so many that
single CTAs serve the batch.  Every call asserts which form ran.  With short ones beside
them each segment has a CTA of its own; with a long one the line is cut inside segments
and their parts are joined."""
import math

import pytest
import torch

import tests.test_gpu_attention as few
from tests.test_gpu_attention import DEV, Case, m  # noqa: F401

pytestmark = pytest.mark.gpu
SHORT = [40, 3, 17, 0, 64, 33, 1, 16]
BESIDE = {"short": SHORT * 5, "long": SHORT * 4 + [4100, 900]}


def _form_ran(c, want, window=0):
    got = c.m.moe_attention_form(c.cache(), len(c.lens), c.q.shape[1], c.table.shape[1], window)
    assert got == want, (got, want)


class InForm(Case):
    """A case that asserts its form and takes its sequences' neighbours from ``beside``."""
    form, beside = "ctas", []

    def __init__(self, m, lens, *a, **kw):  # noqa: F811
        super().__init__(m, [*lens, *self.beside], *a, **kw)

    def cache(self):
        k, v = self.k, self.v  # sizes and order are what the rule looks at
        if self.head_major:
            k, v = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (k, v))
        return self.m.MoeKvCache(k, v, self.ks, self.vs)

    def run(self, window=0, *a, **kw):
        _form_ran(self, self.form, window)
        return super().run(window, *a, **kw)


@pytest.fixture(params=list(BESIDE))
def ctas(request, monkeypatch):
    monkeypatch.setattr(few, "Case", type("Beside", (InForm,), {"beside": BESIDE[request.param]}))


@pytest.mark.parametrize("D", [16, 80, 96, 192, 240])
@pytest.mark.parametrize("e4m3", [False, True])
def test_head_dims_between(m, ctas, D, e4m3):  # noqa: F811
    few.test_head_dims_between(m, D, e4m3)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 20, 32, 48, 64, 128, 1000])
@pytest.mark.parametrize("head_major", [False, True])
def test_page_sizes_and_orders(m, ctas, page, head_major):  # noqa: F811
    few.test_page_sizes_and_orders(m, page, head_major)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (9, 1), (16, 1), (17, 1), (20, 1), (33, 1), (64, 1), (40, 8)])
def test_groups(m, ctas, hq, hkv):  # noqa: F811
    few.test_groups(m, hq, hkv)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 511, 10000])
def test_windows(m, ctas, window):  # noqa: F811
    few.test_windows(m, window)


def test_scale_and_sharp_scores(m, ctas):  # noqa: F811
    few.test_scale_and_sharp_scores(m)


def test_flat_tail_beside_one_large_weight(m, ctas):  # noqa: F811
    few.test_flat_tail_beside_one_large_weight(m)


def test_no_lse(m, ctas):  # noqa: F811
    few.test_no_lse(m)


def test_bad_lengths_are_clamped_and_recorded(m, monkeypatch):  # noqa: F811
    monkeypatch.setattr(few, "Case", type("Beside", (InForm,), {"beside": SHORT[:4] * 10}))
    few.test_bad_lengths_are_clamped_and_recorded(m)


def test_bad_pages_are_dropped_and_recorded(m):  # noqa: F811
    for page, at in ((16, 2), (20, 1), (7, 3)):
        for bad in (-1, -2 ** 31, 2 ** 31 - 1, 100000):
            c = type("Beside", (InForm,), {"beside": BESIDE["long"]})(m, [100, 64], 8, 2, 128, page)
            c.table[0, at] = bad
            c.table[len(c.lens) - 2, 900 // page // 2] = bad
            c.check(status=False)
            with pytest.raises(m.MoeError) as ei:
                m.moe_query_status(c.ws)
            assert ei.value.code == 6 and "page" in str(ei.value)
            m.moe_query_status(c.ws)


def test_non_finite_tokens(m):  # noqa: F811
    for e4m3 in (False, True):
        for beside in BESIDE.values():
            c = type("Beside", (InForm,), {"beside": beside})(m, [100, 64, 30], 8, 2, 128, 16, e4m3=e4m3)
            clean, _ = c.run()
            c.k[int(c.table[0, 1]), 3, 0] = math.nan
            out, _ = c.run()
            assert out[0, :4].isnan().all() and torch.equal(out[0, 4:], clean[0, 4:]) and torch.equal(out[1:], clean[1:])
            win, _ = c.run(window=50)  # outside the window the same token is never read
            assert torch.isfinite(win).all()
            c.v[int(c.table[2, 0]), 3, 1, 7] = math.nan
            out, _ = c.run()
            bad = out[2].isnan()
            assert bad[4:, 7].all() and int(bad.sum()) == 4 and torch.equal(out[3:], clean[3:])


@pytest.mark.parametrize("beside", list(BESIDE))
def test_strided_queries_and_outputs(m, beside):  # noqa: F811
    c = type("Beside", (InForm,), {"beside": BESIDE[beside]})(m, [100, 37], 8, 2, 128, 16)
    B = len(c.lens)
    wide = torch.full((B, 12, 256), 5.0, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 2:10, 64:192]
    q.copy_(c.q)
    out = torch.full((8, B, 192), 5.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    c.check(q=q, out=out[:, :, :128])
    assert (out[:, :, 128:] == 5).all()


@pytest.mark.parametrize("beside", list(BESIDE))
def test_other_stream_graph_and_repeats(m, beside):  # noqa: F811
    c = type("Beside", (InForm,), {"beside": BESIDE[beside]})(m, [700, 33], 8, 2, 128, 20)
    want, lse = c.check()
    ws = c.ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, got_lse = c.run(stream=side, ws=ws)
    assert torch.equal(want, got) and torch.equal(lse, got_lse)
    kd, vd, qd, td = c.k.to(DEV), c.v.to(DEV), c.q.to(DEV), c.table.to(DEV)
    lens = torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    cache = m.MoeKvCache(kd, vd)
    out = torch.empty(c.q.shape, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_paged_attention(cache, qd, td, lens, out, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out.cpu(), want)
    lens.copy_(torch.tensor([1, 20] + c.lens[2:], dtype=torch.int32))  # the same graph serves other lengths
    graph.replay()
    got = out.cpu()
    c.lens = [1, 20] + c.lens[2:]
    want, _ = c.run()
    assert torch.equal(got, want)
    m.moe_query_status(ws)


@pytest.mark.parametrize("window", [300, 777, 1500])
@pytest.mark.parametrize("page", [7, 24])
@pytest.mark.parametrize("D,hq,hkv,dtype,e4m3,head_major", [
    (64, 3, 3, torch.float16, False, False), (128, 10, 2, torch.bfloat16, False, True),
    (96, 24, 2, torch.bfloat16, True, False), (256, 8, 4, torch.bfloat16, False, False)])
def test_windows_on_cut_lines(m, D, hq, hkv, dtype, e4m3, head_major, page, window):  # noqa: F811
    """Windows that begin inside pages and units, over more segments than there are
    workers, so that lines are cut inside them."""
    lens = [3000, 2500, 700, 511, 513, 1501, 0, 1] + [40, 130, 777, 20] * 50
    c = type("Cut", (InForm,), {})(m, lens, hq, hkv, D, page, dtype, e4m3, head_major)
    first, lse = c.check(window)
    again, lse2 = c.run(window, ws=c.ws)
    assert torch.equal(first, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("page", [7, 16, 24])
def test_a_few_long_sequences_in_a_wide_table(m, page):  # noqa: F811
    """The table, not the number of sequences, keeps the teams away."""
    type("Wide", (InForm,), {})(m, [5000, 0, 1, 333, 2048, 77], 8, 2, 128, page, max_pages=3000).check()


@pytest.mark.parametrize("D,hq,hkv,e4m3", [(64, 8, 2, False), (128, 24, 2, True), (256, 8, 1, False)])
def test_both_forms_agree(m, D, hq, hkv, e4m3):  # noqa: F811
    """One batch in a table of its own width and in a wide one, by either form: within
    the bounds each (parts are summed in another order)."""
    for form, width in (("teams", None), ("ctas", 4000)):
        c = type("Form", (InForm,), {"form": form})(m, [900, 31, 0, 517, 64], hq, hkv, D, 16, e4m3=e4m3, max_pages=width)
        c.check()

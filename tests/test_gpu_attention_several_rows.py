"""Several new tokens of one sequence as rows of one call: table rows repeat and lengths
count up, so that each token attends to those before it and itself."""
import pytest
import torch

from tests.test_gpu_attention import Case, m  # noqa: F401

pytestmark = pytest.mark.gpu


def _rows(m, lens, hq, hkv, D, page, dtype, e4m3, max_pages=None):  # noqa: F811
    """Case whose sequences (of (length, new tokens)) have a row per new token."""
    c = Case(m, [n for n, _ in lens], hq, hkv, D, page, dtype, e4m3, max_pages=max_pages)
    row = torch.tensor([b for b, (_, new) in enumerate(lens) for _ in range(new)])
    c.table = c.table[row].contiguous()
    c.lens = [n - new + 1 + i for n, new in lens for i in range(new)]
    c.q = (torch.randn(len(c.lens), hq, D, generator=torch.Generator().manual_seed(9)) * 1.5).to(dtype)
    return c


@pytest.mark.parametrize("dtype,e4m3", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("D,hq,hkv,page", [(64, 8, 8, 7), (128, 8, 2, 16), (256, 16, 2, 16), (128, 24, 2, 20)])
@pytest.mark.parametrize("lens", [[(5, 5)], [(300, 4), (64, 2), (1, 1)], [(700, 40), (33, 33), (90, 3)]])
def test_rows_of_one_sequence(m, lens, D, hq, hkv, page, dtype, e4m3):  # noqa: F811
    c = _rows(m, lens, hq, hkv, D, page, dtype, e4m3)
    c.check()
    c.check(window=13)


def test_each_row_equals_its_own_call(m):  # noqa: F811
    """A chunk's rows are what single calls give one after the other, within both bounds."""
    c = _rows(m, [(400, 9)], 8, 2, 128, 16, torch.bfloat16, False)
    c.check()
    q, lens, table = c.q, c.lens, c.table
    for i in range(0, 9, 4):
        c.q, c.lens, c.table = q[i:i + 1], lens[i:i + 1], table[i:i + 1].contiguous()
        c.check()


def test_a_chunk_appended_and_attended(m):  # noqa: F811
    """New tokens rotated by nothing (no frequencies), appended in one call and attended
    in the next, without anything between the two."""
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(2)
    T, hq, hkv, D, P = 21, 8, 2, 64, 8
    q, k, v = ((torch.randn(T, h, D, generator=g)).to(torch.bfloat16) for h in (hq, hkv, hkv))
    kc, vc = (torch.zeros(5, P, hkv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    cache = m.MoeKvCache(kc, vc)
    ws = m.alloc_attention_workspace(cache, hq)
    pages = torch.tensor([3, 0, 4], dtype=torch.int32)
    t = torch.arange(T)
    slots = pages.long()[t // P] * P + t % P
    table = pages.expand(T, 3).contiguous().to(dev)
    lens = (t + 1).to(torch.int32).to(dev)
    out = torch.empty(T, hq, D, dtype=torch.bfloat16, device=dev)
    qd, kd, vd, qo = q.to(dev), k.to(dev), v.to(dev), torch.empty(T, hq, D, dtype=torch.bfloat16, device=dev)
    args = (t.to(dev), slots.to(dev), torch.empty(0, device=dev))
    torch.cuda.synchronize()
    m.moe_rope_append(cache, qd, kd, vd, *args, qo, ws)
    m.moe_paged_attention(cache, qo, table, lens, out, ws)
    m.moe_query_status(ws)
    assert torch.equal(qo.cpu(), q)
    c = Case.__new__(Case)
    c.m, c.lens, c.dtype, c.e4m3, c.ks, c.vs, c.head_major = m, [i + 1 for i in range(T)], torch.bfloat16, False, None, None, False
    c.q, c.table, c.k, c.v = q, table.cpu(), kc.cpu(), vc.cpu()
    want, _ = c.check()
    assert torch.equal(out.cpu(), want)

"""Infinite values in the cache: a token with a positive weight makes the output's
column infinite with the value's sign, infinities of both signs make it NaN, and
all other columns, heads and sequences keep what they are without them."""
import math

import pytest
import torch

from tests.test_gpu_attention import Case, m  # noqa: F401

pytestmark = pytest.mark.gpu
INF = math.inf
# up to 32 short sequences go to teams of CTAs, more to single ones
LENS = {"teams": [100, 64, 30], "ctas": [100, 64, 30] * 14, "long": [6001, 64, 30] * 14}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 2), (64, 24, 2), (128, 16, 2), (256, 8, 1), (256, 20, 2)])
@pytest.mark.parametrize("form", list(LENS))
def test_infinite_values_stay_infinite(m, form, D, hq, hkv, dtype):  # noqa: F811
    G = hq // hkv
    # scores of small spread: no weight is lost beside the largest
    c = Case(m, LENS[form], hq, hkv, D, 16, dtype, q_scale=0.5)
    clean, lse = c.check()
    put = [(0, 3, 5, INF), (0, 70, 6, -INF), (0, 17, 7, INF), (0, 40, 7, -INF), (0, 9, 8, INF), (0, 90, 8, INF),
           (1, 63, 5, -INF)]
    for b, tok, col, value in put:  # of the first kv head
        c.v[int(c.table[b, tok // 16]), tok % 16, 0, col] = value
    want = clean.clone()
    want[0, :G, 5], want[0, :G, 6], want[0, :G, 7], want[0, :G, 8] = INF, -INF, math.nan, INF
    want[1, :G, 5] = -INF
    out, lse2 = c.run()
    assert torch.equal(lse, lse2)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(nan=0.0, posinf=3e4, neginf=-3e4), want.nan_to_num(nan=0.0, posinf=3e4, neginf=-3e4))


def test_finite_values_of_the_largest_size(m):  # noqa: F811
    """The largest finite values are no infinities: one token's value comes back as it
    is, and sums that fp32 holds are finite."""
    big = torch.finfo(torch.bfloat16).max
    c = Case(m, [1, 50, 33], 4, 1, 64, 16, q_scale=0.5)
    c.v.fill_(big / 64)
    c.v[:, :, :, 1] = -big / 64
    c.v[int(c.table[0, 0]), 0, 0, :3] = torch.tensor([big, -big, INF])
    c.v[int(c.table[1, 1]), 2, 0, 9] = -INF
    out, _ = c.run()
    assert (out[0, :, 0] == big).all() and (out[0, :, 1] == -big).all() and (out[0, :, 2] == INF).all()
    assert (out[1, :, 9] == -INF).all()
    c.v[int(c.table[0, 0]), 0, 0, 2] = 0.0
    c.v[int(c.table[1, 1]), 2, 0, 9] = 0.0
    c.check()

"""The norm's refusal of outputs that lie on rows other rows still have to read, before
anything touches a GPU.  Rows are told by address, distance and width in bytes."""
import pytest
import torch

from tests.test_layer_host import NORM, m  # noqa: F401

# (the addresses are made up, so what a mistake would let through has to find no GPU)
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="calls with made-up addresses")
FAR = 1 << 20


def _call(m, **kw):  # noqa: F811
    """A call whose tensors are apart unless told otherwise."""
    a = {**NORM, "x": FAR, "residual": 2 * FAR, "out": 3 * FAR, "residual_out": 4 * FAR, "T": 4, **kw}
    return m.library().moe_add_rmsnorm(m._NORM_T.pack(*a.values()), None)


def _e4m3(**kw):
    return {"out_dtype": 4, "scales": 5 * FAR, **kw}


@pytest.mark.parametrize("change", [
    _e4m3(out=FAR),                                    # in place, rows of out at half the distance of x's
    _e4m3(out=2 * FAR),                                # the same over the residual
    _e4m3(out=FAR + 3 * 128 + 64, os=192),             # only x's last row, from another row
    dict(out=FAR, os=72),                              # in place with other strides
    dict(out=FAR + 128),                               # a row behind
    dict(out=FAR - 128),                               # a row ahead
    dict(out=FAR + 64),                                # half a row behind: the next one's first half
    dict(residual_out=FAR + 256),
    dict(residual_out=2 * FAR, ros=80),
    dict(residual_out=2 * FAR - 384 + 2),
    dict(out=FAR, residual_out=FAR),                   # two outputs in one place
    dict(out=4 * FAR + 3 * 128 + 126),
    dict(out=4 * FAR + 130, T=2, H=64),
    dict(out=4 * FAR, T=1),                            # ... where one row is all there is, too
])
def test_outputs_on_other_rows_are_refused(m, change):  # noqa: F811
    assert _call(m, **change) == 1, m.moe_last_error()
    assert "overlap" in m.moe_last_error()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 2, 4])
@pytest.mark.parametrize("H,stride", [(8, 8), (5, 5), (5, 8), (8, 11)])
def test_the_rule_against_every_byte(m, H, stride, T, e4m3):  # noqa: F811
    """Rows at one distance in bytes: refused exactly where a row's output shares a byte
    with another row's input.  (What passes the checks fails to launch here.)"""
    step, n_out = 2 * stride, H if e4m3 else 2 * H
    kw = dict(T=T, H=H, xs=stride, rs=stride, ros=stride, os=step if e4m3 else stride)
    if e4m3:
        kw.update(_e4m3())
    for q in range(FAR - 5 * step, FAR + 5 * step, 1 if e4m3 else 2):
        shared = any(set(range(FAR + i * step, FAR + i * step + 2 * H)) & set(range(q + j * step, q + j * step + n_out))
                     for i in range(T) for j in range(T) if i != j)
        rc = _call(m, out=q, **kw)
        assert rc == 1 if shared else rc not in (0, 1, 2, 3), (q - FAR, m.moe_last_error())

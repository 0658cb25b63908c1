"""Compiled argument checks of the quantisation, the 8-bit product and the drawing of
tokens that are missing or of other structs are named, and not used."""
import types
import warnings

import pytest
import torch

from tests.test_layer_host import m  # noqa: F401


@pytest.mark.parametrize("other", [dict(), dict(bind_projections=lambda *a: False)])
def test_missing_or_refused(m, monkeypatch, other):  # noqa: F811
    module = types.SimpleNamespace(built_for=torch.__version__, bind=lambda *a: True, **other)
    monkeypatch.setattr(m, "_fast", None)
    monkeypatch.setattr(m, "_fast_projections", None)
    monkeypatch.setattr(m, "_fast_call", module, raising=False)
    with pytest.warns(UserWarning, match="8-bit projections"):
        m._bind_fast_call(m.library())
    assert m._fast is module and m._fast_projections is None


def test_bound_without_a_word(m, monkeypatch):  # noqa: F811
    module = types.SimpleNamespace(built_for=torch.__version__, bind=lambda *a: True, bind_projections=lambda *a: True)
    monkeypatch.setattr(m, "_fast", None)
    monkeypatch.setattr(m, "_fast_projections", None)
    monkeypatch.setattr(m, "_fast_call", module, raising=False)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        m._bind_fast_call(m.library())
    assert m._fast is module and m._fast_projections is module


def test_the_module_refuses_structs_of_other_sizes(m):  # noqa: F811
    fast = pytest.importorskip("moe_decode_expert_gb300._fast_call")
    sizes = [t.size for t in (m._QUANT_T, m._LINEAR_T, m._SAMPLING_T)]
    for i in range(3):
        wrong = [s + 8 * (i == j) for j, s in enumerate(sizes)]
        assert fast.bind_projections(0, 0, 0, *wrong) is False
    assert fast is m._fast_projections

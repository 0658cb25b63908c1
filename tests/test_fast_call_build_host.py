"""The compiled argument checks are used only with the PyTorch, interpreter and structs
they were compiled for, and no older module stays where compiling fails."""
import os
import subprocess
import types

import pytest
import torch

from tests.test_layer_host import m  # noqa: F401


@pytest.fixture
def place(tmp_path, monkeypatch):
    """build_fast_call in a folder of its own, with a compiler that the test plays."""
    from moe_decode_expert_gb300 import _build
    monkeypatch.setattr(_build, "FAST_CALL", str(tmp_path / os.path.basename(_build.FAST_CALL)))
    monkeypatch.setattr(_build, "FAST_CALL_KEY", str(tmp_path / "key" / "fast_call.key"), raising=False)
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("compiled")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(_build.subprocess, "run", compiler)
    return _build, runs


def test_compiled_once_for_one_pytorch(place, monkeypatch):
    b, runs = place
    assert b.build_fast_call() == b.FAST_CALL and b.build_fast_call() == b.FAST_CALL and len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert b.build_fast_call() == b.FAST_CALL and len(runs) == 2
    assert b.build_fast_call() == b.FAST_CALL and len(runs) == 2
    os.remove(b.FAST_CALL_KEY)
    assert b.build_fast_call() == b.FAST_CALL and len(runs) == 3


@pytest.mark.parametrize("how", ["absent", "failing"])
def test_a_failed_build_leaves_no_older_module(place, monkeypatch, capsys, how):
    b, _ = place
    old = os.path.join(os.path.dirname(b.FAST_CALL), "_fast_call.so")
    for f in (b.FAST_CALL, old):
        with open(f, "w") as out:
            out.write("older")
        os.utime(f, (0, 0))

    def compiler(cmd, **kw):
        if how == "absent":
            raise FileNotFoundError(cmd[0])
        return subprocess.CompletedProcess(cmd, 1, "", "no such header")

    monkeypatch.setattr(b.subprocess, "run", compiler)
    assert b.build_fast_call() is None
    assert not os.path.exists(b.FAST_CALL) and not os.path.exists(old)
    assert "not built" in capsys.readouterr().err


def test_the_name_tells_the_interpreter():
    from moe_decode_expert_gb300 import _build
    import sysconfig
    assert _build.FAST_CALL.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_a_module_for_another_pytorch_or_other_structs_is_not_used(m, monkeypatch):  # noqa: F811
    lib = m.library()
    monkeypatch.setattr(m, "_fast", None)
    ours = dict(built_for=torch.__version__, bind=lambda *a: True)
    for other in (dict(ours, built_for="0.0.1"), dict(bind=ours["bind"]), dict(ours, bind=lambda *a: False)):
        monkeypatch.setattr(m, "_fast_call", types.SimpleNamespace(**other), raising=False)
        with pytest.warns(UserWarning, match="built"):
            m._bind_fast_call(lib)
        assert m._fast is None
    same = types.SimpleNamespace(**ours)
    monkeypatch.setattr(m, "_fast_call", same, raising=False)
    m._bind_fast_call(lib)
    assert m._fast is same


def test_the_module_refuses_structs_of_other_sizes(m):  # noqa: F811
    fast = pytest.importorskip("moe_decode_expert_gb300._fast_call")
    sizes = [t.size for t in (m._NORM_T, m._CACHE_T, m._ROPE_T, m._ATTN_T)]
    assert fast.built_for == torch.__version__
    for i in range(4):
        wrong = [s + 8 * (i == j) for j, s in enumerate(sizes)]
        assert fast.bind(0, 0, 0, *wrong) is False
    assert fast is m._fast

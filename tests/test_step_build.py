"""The module of ordinary calls is compiled for one torch and serves no other (no GPU, no compiler: the compile command is counted)."""
import os
import subprocess
import types

import pytest


@pytest.fixture
def b(tmp_path, monkeypatch):
    from w4a16_int4_weight_group_gb300 import build
    state = types.SimpleNamespace(build=build, commands=[], status=0)

    def run(cmd, **kw):
        state.commands.append(cmd)
        if state.status == 0:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("module")
        return types.SimpleNamespace(returncode=state.status, stdout="", stderr="no")

    monkeypatch.setattr(build, "FAST_PATH", str(tmp_path / "fast.so"))
    monkeypatch.setattr(build, "FAST_STAMP", str(tmp_path / "_build" / "fast.key"), raising=False)
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(subprocess, "run", run)
    if not build.build_fast():
        pytest.skip("no compiler, headers or CUDA toolkit")
    return state


def another_torch(monkeypatch):
    import torch
    monkeypatch.setattr(torch, "__version__", "2.99.0")


def test_it_is_compiled_again_for_another_torch(b, monkeypatch):
    assert len(b.commands) == 1 and b.build.build_fast() and len(b.commands) == 1
    another_torch(monkeypatch)
    assert b.build.build_fast() and len(b.commands) == 2
    assert any("2.99.0" in x for x in b.commands[1])
    assert b.build.build_fast() and len(b.commands) == 2
    os.remove(b.build.FAST_PATH)
    assert b.build.build_fast() and len(b.commands) == 3


def test_what_cannot_be_compiled_is_said_and_not_tried_again(b, monkeypatch, capsys):
    another_torch(monkeypatch)
    b.status = 1
    assert not b.build.build_fast() and len(b.commands) == 2
    assert "could not be compiled" in capsys.readouterr().err
    assert not b.build.build_fast() and len(b.commands) == 2
    b.status = 0
    assert b.build.build_fast(force=True) and len(b.commands) == 3


def test_a_module_for_another_torch_is_not_used(monkeypatch):
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    from w4a16_int4_weight_group_gb300 import step
    monkeypatch.setattr(step, "_fast", None)
    if not step._bind_fast():
        pytest.skip("the module of ordinary calls was not built")
    another_torch(monkeypatch)
    assert step._bind_fast() is False

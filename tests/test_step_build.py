"""The binding module _step.so is built for one torch and one Python: it is built anew,
or refused, when either has changed. The compiler and the module are stand-ins.
"""
import os
import subprocess
import types

import pytest

from latent_kv_decode_b200 import build, ops


@pytest.fixture
def fake(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "STEP", str(tmp_path / "_step.so"))
    monkeypatch.setattr(build, "STEP_STAMP", str(tmp_path / "step.built_for"))
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    return runs


def test_built_once_and_again_for_another_torch(fake, monkeypatch):
    build.build_step()
    build.build_step()
    assert len(fake) == 1
    assert any(build.built_for() in a for a in fake[0])
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build_step()
    build.build_step()
    assert len(fake) == 2 and any("torch 0.0.1" in a for a in fake[1])


def test_built_again_without_a_record_of_what_it_was_built_for(fake):
    build.build_step()
    os.remove(build.STEP_STAMP)
    build.build_step()
    assert len(fake) == 2


def test_a_module_of_another_torch_is_refused(monkeypatch):
    if not os.path.exists(ops.STEP_PATH):
        build.build()
    monkeypatch.setattr(ops, "_step_mod", None)
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ops.MlaError, match="built for"):
        ops._step()
    assert ops._step_mod is None


def test_a_module_that_does_not_load_is_refused(tmp_path, monkeypatch):
    bad = tmp_path / "_step.so"
    bad.write_bytes(b"not a module")
    monkeypatch.setattr(ops, "STEP_PATH", str(bad))
    monkeypatch.setattr(ops, "_step_mod", None)
    with pytest.raises(ops.MlaError, match="does not load"):
        ops._step()

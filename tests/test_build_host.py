"""What a build needs, and when the torch binding is built again (no GPU, and no compiler run here)."""
import os
import sys

import pytest

import linear_attention_sequence_chunkwise_b200 as rn
from linear_attention_sequence_chunkwise_b200 import _build


@pytest.fixture()
def apart(tmp_path, monkeypatch):
    """A built library, and a place of its own for the binding; what would be compiled is recorded."""
    _build.build()
    lib, binding = tmp_path / "libretnet.so", tmp_path / "_torch_binding.so"
    lib.touch()
    monkeypatch.setattr(_build, "LIB", str(lib))
    monkeypatch.setattr(_build, "BINDING", str(binding))
    monkeypatch.setattr(_build, "BINDING_KEY", str(tmp_path / "key"), raising=False)
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    ran = []

    def run(cmd, check):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
    monkeypatch.setattr(_build.subprocess, "run", run)
    return binding, ran


def test_the_library_is_built_without_torch(apart, monkeypatch, capsys):
    binding, ran = apart
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch: ImportError
    assert _build.build() == _build.LIB
    assert not ran and not binding.exists()
    assert "torch binding is not" in capsys.readouterr().err


def test_the_binding_is_built_again_for_another_torch_or_python(apart, monkeypatch):
    binding, ran = apart
    _build.build()
    assert len(ran) == 1 and binding.exists()
    _build.build()
    assert len(ran) == 1  # nothing changed
    import torch
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    _build.build()
    assert len(ran) == 2
    monkeypatch.undo()


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    _build.build()
    monkeypatch.setattr(rn, "_binding", None)
    assert rn._native().built_for == _build.binding_key()
    monkeypatch.setattr(rn, "_binding", None)
    monkeypatch.setattr(_build, "binding_key", lambda: "torch 9.9.9")
    with pytest.raises(RuntimeError, match="build it again"):
        rn._native()
    monkeypatch.undo()
    monkeypatch.setattr(rn, "_binding", None)
    monkeypatch.delitem(sys.modules, rn.__name__ + "._torch_binding", raising=False)
    monkeypatch.delattr(rn, "_torch_binding", raising=False)
    monkeypatch.setattr(rn, "__path__", [os.devnull])
    with pytest.raises(RuntimeError, match="missing"):
        rn._native()

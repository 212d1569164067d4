"""What is built when: the library without torch, the binding for the Python
and the torch that are there."""
import importlib.util

import pytest

from int8_conv2d_fprop_gb300 import _build


@pytest.fixture
def built(monkeypatch, tmp_path):
    """Names of what build() makes, which here makes nothing."""
    made = []
    binding = tmp_path / "_channel.so"
    monkeypatch.setattr(_build, "BINDING", str(binding))
    monkeypatch.setattr(_build, "BINDING_STAMP", str(tmp_path / "channel_binding.txt"), raising=False)
    monkeypatch.setattr(_build, "build_library", lambda *a, **k: made.append("library"))

    def run(cmd, **kwargs):
        made.append("binding")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return type("Done", (), {"returncode": 0, "stderr": ""})

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return made


def test_the_library_builds_without_torch(built, monkeypatch, capsys):
    import builtins
    real, real_import = importlib.util.find_spec, builtins.__import__

    def no_torch(name, *a, **k):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'")
        return real_import(name, *a, **k)

    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert _build.build() == _build.LIB
    assert built == ["library"]
    assert "torch" in capsys.readouterr().err


def test_the_binding_is_built_again_for_another_torch_or_python(built, monkeypatch):
    pytest.importorskip("torch")
    _build.build()
    _build.build()
    assert built == ["library", "binding", "library"]  # the second time it was there
    with open(_build.BINDING_STAMP) as f:
        target = f.read()
    for other in (target.replace("__version__", "__version__ = '0.0' #"), "another Python\n" + target):
        assert other != target
        with open(_build.BINDING_STAMP, "w") as f:
            f.write(other)
        del built[:]
        _build.build()
        _build.build()
        assert built == ["library", "binding", "library"]

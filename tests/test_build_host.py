"""The build of the library and of the recurrent layer's binding, with commands
that only write their outputs: libvdc.so needs no torch and comes before
anything of the binding can fail."""
import importlib.util
import subprocess

import pytest

from varlen_depthwise_causal_amd import _build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """Compilers and linkers that write what -o names, or fail for a source in
    `failing`; returns the outputs in the order in which they were written."""
    made, failing = [], []

    class Compiler:
        def __init__(self, cmd, **_):
            self.args = cmd
            self.returncode = 1 if any(f in a for f in failing for a in cmd) else 0
            if not self.returncode:
                out = cmd[cmd.index("-o") + 1]
                open(out, "w").close()
                made.append(out)

        def wait(self, timeout=None):
            return self.returncode

        poll = wait

        def communicate(self, *_, **__):
            return None, None

        def __enter__(self):
            return self

        def __exit__(self, *_):
            return False

    monkeypatch.setattr(subprocess, "Popen", Compiler)
    monkeypatch.setattr(_build, "hipcc", lambda: "/opt/rocm/bin/hipcc")
    for name, at in (("BUILD_DIR", "build"), ("LIBRARY", "libvdc.so"), ("BINDING", "_vdc_torch.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / at))
    return made, failing


def there(tmp_path):
    return {n for n in ("libvdc.so", "_vdc_torch.so") if (tmp_path / n).exists()}


def test_both(commands, tmp_path):
    assert _build.build() == str(tmp_path / "libvdc.so")
    assert there(tmp_path) == {"libvdc.so", "_vdc_torch.so"}


def test_the_library_needs_no_torch(commands, tmp_path, monkeypatch, capsys):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    assert _build.build() == str(tmp_path / "libvdc.so")
    assert there(tmp_path) == {"libvdc.so"}
    assert "torch not found" in capsys.readouterr().out


@pytest.mark.parametrize("part", ["vdc_torch.cpp", "-ltorch_cpu"])
def test_a_binding_that_fails_comes_after_the_library(commands, tmp_path, part):
    commands[1].append(part)
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert there(tmp_path) == {"libvdc.so"}


def test_a_library_that_fails_is_the_end(commands, tmp_path):
    commands[1].append("vdc_pool.hip")
    with pytest.raises(subprocess.CalledProcessError):
        _build.build()
    assert there(tmp_path) == set()

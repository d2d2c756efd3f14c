"""What a build makes where something it would use is not there."""
import os
import sysconfig

import pytest

import calibration_free_channel_amd.build as b


@pytest.fixture
def dry(tmp_path, monkeypatch):
    """build() into an empty folder, with compilers that only make their output."""
    made = []

    def run(cmd, verbose):
        if any("py_ops.cpp" in c for c in cmd):
            include = [c[2:] for c in cmd if c.startswith("-I")]
            if not any(os.path.exists(os.path.join(d, "Python.h")) for d in include):
                raise RuntimeError("build step failed: Python.h: No such file or directory")
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out))
    for name, file in (("LIB", "libcfr.so"), ("OPS", "_ops.so"), ("BUILD", "_build")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    monkeypatch.setattr(b, "_run", run)
    return made


def test_everything_is_built(dry):
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and os.path.exists(b.OPS)


def test_library_is_built_without_pythons_headers(dry, tmp_path, monkeypatch, capsys):
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    open(b.OPS, "w").close()  # of an earlier build: it may not fit this library
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.OPS)
    assert "Python.h" in capsys.readouterr().out


def test_library_is_built_without_torch(dry, monkeypatch, capsys):
    import builtins
    real = builtins.__import__

    def no_torch(name, *a, **k):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError(f"No module named {name!r}", name=name)
        return real(name, *a, **k)
    monkeypatch.setattr(builtins, "__import__", no_torch)
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.OPS)
    assert "torch" in capsys.readouterr().out

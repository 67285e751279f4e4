"""The build: the C library needs nvcc alone; the torch extension comes with torch and goes with its version."""

import os
import sys

import pytest

from conftest import load_build_module


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build module on an empty output folder, its commands recorded instead of run."""
    b = load_build_module()
    pkg = tmp_path / "pkg"
    pkg.mkdir()
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(pkg / "libsplitkv.so"))
    monkeypatch.setattr(b, "EXT", str(pkg / "_draft_ext.so"))
    ran = []

    class Done:
        returncode, stderr, stdout = 0, "", ""

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return Done()

    monkeypatch.setattr(b.subprocess, "run", run)
    return b, ran


def _ext(ran, b):
    return [c for c in ran if b.EXT in c]


def test_the_library_builds_without_torch(tree, monkeypatch, capsys):
    b, ran = tree
    monkeypatch.setitem(sys.modules, "torch", None)          # `import torch` raises ImportError
    monkeypatch.setattr(b, "_torch_version", lambda: None, raising=False)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not _ext(ran, b) and not os.path.exists(b.EXT)
    assert "_draft_ext.so" in capsys.readouterr().err        # said, not silent


def test_the_extension_is_built_once_per_torch(tree, monkeypatch):
    b, ran = tree
    b.build()
    assert len(_ext(ran, b)) == 1
    b.build()
    assert len(_ext(ran, b)) == 1
    monkeypatch.setattr(b, "_torch_version", lambda: "99.0", raising=False)
    b.build()
    assert len(_ext(ran, b)) == 2
    b.build()
    assert len(_ext(ran, b)) == 2
    os.remove(b.EXT)
    b.build()
    assert len(_ext(ran, b)) == 3


def test_a_failed_extension_build_is_an_error(tree, monkeypatch):
    b, _ = tree
    inner = b.subprocess.run

    def run(cmd, **kw):
        if b.EXT in cmd:
            raise b.subprocess.CalledProcessError(1, cmd)
        return inner(cmd, **kw)

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.raises(b.subprocess.CalledProcessError):
        b.build()
    with pytest.raises(b.subprocess.CalledProcessError):     # and is tried again
        b.build()

"""The in-tree build on the host: a marshalling module that cannot be rebuilt
does not stay behind for the binding to load."""
import subprocess

import pytest

from sparse_paged_decode_gb300 import build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A module of earlier sources, in a folder of its own."""
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    (tmp_path / "_marshal.so").write_bytes(b"earlier")
    (tmp_path / "marshal.stamp").write_text("of other sources")
    return tmp_path


def refused(cmd, **_):
    return subprocess.CompletedProcess(cmd, 1, "", "error: no")


def absent(cmd, **_):
    raise FileNotFoundError(cmd[0])


@pytest.mark.parametrize("compiler", [refused, absent])
def test_a_module_that_cannot_be_rebuilt_is_removed(built, monkeypatch, compiler):
    monkeypatch.setattr(subprocess, "run", compiler)
    assert build.build_marshal() is False
    assert not (built / "_marshal.so").exists() and not (built / "marshal.stamp").exists()
    assert build.build_marshal() is False  # nothing to remove


def test_a_module_is_rebuilt_once(built, monkeypatch):
    calls = []

    def compiles(cmd, **_):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"new")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", compiles)
    for _ in range(2):
        assert build.build_marshal() is True
        assert (built / "_marshal.so").read_bytes() == b"new"
    assert len(calls) == 1

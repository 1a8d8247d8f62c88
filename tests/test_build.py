"""What the build needs, and when it builds the extension module again (no GPU)."""
import os
import subprocess
import sys

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build of an extension in another place, beside the library that is there."""
    import __graft_entry__ as g
    g.build()
    from sparse_moe_decode_gb300 import build as b
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "BINDING_STAMP", str(tmp_path / "x" / "binding.txt"), raising=False)
    return b


def test_library_is_built_without_torch(build, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING) and "torch" in capsys.readouterr().err


def test_library_is_built_without_a_host_compiler_of_its_own(build, monkeypatch, capsys):
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING) and "no-such-compiler" in capsys.readouterr().err


def test_errors_in_the_source_are_raised(build, monkeypatch, tmp_path):
    bad = tmp_path / "bad.cpp"
    bad.write_text("this is not C++\n")
    monkeypatch.setattr(build, "BINDING_SRC", str(bad))
    with pytest.raises(RuntimeError, match="bad.cpp"):
        build.build()


def test_extension_is_built_again_for_another_torch(build, monkeypatch):
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    for target, count in (("one", 1), ("one", 1), ("two", 2), ("two", 2)):
        monkeypatch.setattr(build, "binding_target", lambda: target, raising=False)
        assert build.build_binding() == build.BINDING
        assert len(runs) == count
    os.remove(build.BINDING)
    build.build_binding()
    assert len(runs) == 3

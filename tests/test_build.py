"""The build with its compilers stubbed: the library needs hipcc alone, the C++ marshalling of the linear layer is left out
where it cannot be built, and a failed compiler is named."""
import os
import sys

import pytest

from async_stage_tile_amd import build


@pytest.fixture
def stubbed(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_linear.so"))
    monkeypatch.setattr(build, "hipcc", lambda: "hipcc")
    commands = []

    def run(cmd, verbose):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(build, "_run", run)
    return commands


def test_library_and_binding(stubbed):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
    assert len(stubbed) == len(build.UNITS) + 2     # the objects, the link, the binding


@pytest.mark.parametrize("reason", [ModuleNotFoundError("No module named 'torch'"), RuntimeError("g++ failed")])
def test_library_without_the_binding(stubbed, monkeypatch, capsys, reason):
    with open(build.BINDING, "w") as f:
        f.write("of an earlier build")

    def fails(verbose=False):
        raise reason

    monkeypatch.setattr(build, "build_binding", fails)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING)
    assert str(reason) in capsys.readouterr().err


def test_failed_compiler_and_source_are_named(capsys):
    with pytest.raises(RuntimeError, match=r"python.* failed with exit code 3: some\.cpp"):
        build._run([sys.executable, "-c", "raise SystemExit(3)", "some.cpp", "-o", "x"], False)

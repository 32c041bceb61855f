"""CPU tests of the build's order: nothing is put in place before everything is
whole, and the collectives' library needs no torch.  The compilers are small
scripts that write their output file."""

import os
import sys

import pytest

from tree_allreduce_algorithms_amd import build_lib


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """A package folder with old results, and compilers that fail on demand."""
    script = "import os, sys\nif os.environ.get('BREAK') == '{0}': sys.exit('broken {0}')\n" \
             "open(sys.argv[sys.argv.index('-o') + 1], 'w').write('new {0}')\n"
    for name in ("hipcc", "g++"):
        path = tmp_path / name
        path.write_text(f"#!{sys.executable}\n" + script.format(name))
        path.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(tmp_path / "hipcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "g++"))
    monkeypatch.setattr(build_lib, "LIB", str(tmp_path / "libar.so"))
    monkeypatch.setattr(build_lib, "MODULE", str(tmp_path / "_training.so"))
    for path in (build_lib.LIB, build_lib.MODULE):
        open(path, "w").write("old")
    return lambda: (open(build_lib.LIB).read(), open(build_lib.MODULE).read())


def test_both_are_put_in_place(tools):
    assert build_lib.build() == build_lib.LIB
    assert tools() == ("new hipcc", "new g++")


@pytest.mark.parametrize("broken", ["hipcc", "g++"])
def test_a_failure_leaves_both_as_they_were(tools, monkeypatch, broken):
    monkeypatch.setenv("BREAK", broken)
    with pytest.raises(RuntimeError, match="failed"):
        build_lib.build()
    assert tools() == ("old", "old")


def test_the_library_is_built_without_torch(tools, monkeypatch, capsys):
    monkeypatch.setattr(build_lib, "has_torch", lambda: False)
    build_lib.build()
    assert tools() == ("new hipcc", "old")
    assert "torch is not installed" in capsys.readouterr().err


def test_hipccs_own_compiler_serves_where_there_is_no_other(monkeypatch):
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setenv("PATH", "/nowhere")
    monkeypatch.delenv("HIPCC", raising=False)
    assert os.path.exists(build_lib.host_compiler())

"""What build() does when part of its tools is missing, with compilers that only leave a file (no GPU)."""
import os
import stat
import sys

import pytest

from draft_tree_construction_gb300 import _build

WORKS = """#!{python}
import sys
open({log!r}, "a").write(" ".join(sys.argv) + "\\n")
open(sys.argv[sys.argv.index("-o") + 1], "w").write("made")
"""
FAILS = """#!{python}
import sys
open({log!r}, "a").write(" ".join(sys.argv) + "\\n")
sys.exit("no such header")
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() on targets of its own; set("NVCC" or "CXX", works) replaces a compiler, calls() counts its runs."""
    def setup(tool, text):
        path, log = tmp_path / tool, tmp_path / f"{tool}.log"
        path.write_text(text.format(python=sys.executable, log=str(log)))
        path.chmod(path.stat().st_mode | stat.S_IXUSR)
        monkeypatch.setattr(_build, tool, str(path))
    for name, target in (("LIB", "lib.so"), ("BUILD", "objects")):
        monkeypatch.setattr(_build, name, str(tmp_path / target))
    monkeypatch.setattr(_build, "native_path", lambda: str(tmp_path / "native.so"))
    monkeypatch.setattr(_build, "_native_failed", False, raising=False)
    setup("NVCC", WORKS)
    setup("CXX", WORKS)
    t = type("Tree", (), {})()
    t.set = setup
    t.calls = lambda tool: len((tmp_path / f"{tool}.log").read_text().splitlines()) if (
        tmp_path / f"{tool}.log").exists() else 0
    t.files = lambda: {f for f in os.listdir(tmp_path) if ".so" in f}
    return t


def test_both_are_built_once(tree):
    assert _build.needs_build()
    assert _build.build() == _build.LIB
    assert tree.files() == {"lib.so", "native.so"} and not _build.needs_build()
    assert (tree.calls("NVCC"), tree.calls("CXX")) == (len(_build.SOURCES) + 1, 1)
    _build.build()
    assert (tree.calls("NVCC"), tree.calls("CXX")) == (len(_build.SOURCES) + 1, 1)
    _build.build(force=True)
    assert (tree.calls("NVCC"), tree.calls("CXX")) == (2 * len(_build.SOURCES) + 2, 2)


def test_the_library_is_linked_without_the_module(tree):
    tree.set("CXX", FAILS)
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert _build.build() == _build.LIB
    assert tree.files() == {"lib.so"}
    assert not _build.needs_build()
    _build.build()                                   # said once, tried once
    assert (tree.calls("NVCC"), tree.calls("CXX")) == (len(_build.SOURCES) + 1, 1)


def test_the_library_is_linked_without_a_host_compiler_or_pytorch(tree, monkeypatch):
    def missing(target):
        raise ModuleNotFoundError("No module named 'torch'")
    monkeypatch.setattr(_build, "_native_command", missing)
    with pytest.warns(RuntimeWarning, match="No module named"):
        _build.build()
    assert tree.files() == {"lib.so"} and tree.calls("CXX") == 0


def test_a_library_that_fails_to_compile_raises(tree):
    tree.set("NVCC", FAILS)
    with pytest.raises(RuntimeError, match="no such header"):
        _build.build()
    assert "lib.so" not in tree.files() and _build.needs_build()


def test_a_compiler_that_dies_without_a_word_has_failed(tree, tmp_path):
    tree.set("CXX", "#!{python}\nimport sys\n# {log}\nopen(sys.argv[sys.argv.index('-o') + 1], 'w')\nsys.exit(9)\n")
    with pytest.warns(RuntimeWarning, match="returned 9"):
        _build.build()
    assert tree.files() == {"lib.so"}


def test_a_failed_build_leaves_no_parts(tree):
    tree.set("NVCC", FAILS)
    with pytest.raises(RuntimeError):
        _build.build()
    assert tree.files() == set()


def test_a_module_of_other_sources_does_not_stay(tree):
    """Its structures may lie differently than the new library's."""
    _build.build()
    tree.set("CXX", FAILS)
    with pytest.warns(RuntimeWarning):
        _build.build(force=True)
    assert tree.files() == {"lib.so"}


def test_the_module_is_one_for_each_pytorch_and_interpreter(tree, tmp_path, monkeypatch):
    """After an upgrade the module of the versions before is neither taken for fresh nor loaded."""
    import sysconfig

    torch = pytest.importorskip("torch")
    monkeypatch.undo()
    own = _build.native_path()
    assert torch.__version__ in own and own.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    other = _build.native_path()
    assert other != own and os.path.dirname(other) == _build.HERE and not os.path.exists(other)
    assert _build.needs_build() and _build._native_stale()


def test_modules_of_an_older_library_go_with_it(tree, tmp_path, monkeypatch):
    monkeypatch.setattr(_build, "native_path", lambda: str(tmp_path / "_steps_native.two.so"))
    (tmp_path / "_steps_native.one.so").write_text("of another PyTorch")
    _build.build()
    assert tree.files() == {"lib.so", "_steps_native.two.so"}
    (tmp_path / "_steps_native.one.so").write_text("of another PyTorch")
    _build.build()                                   # the library stays, and so does what was built for it
    assert tree.files() == {"lib.so", "_steps_native.one.so", "_steps_native.two.so"}

"""The compiled argument checks are optional: the library is built without them, what an earlier
build left does not stay, and a module made for something else is not taken."""
import os
import sys
import types

import pytest

import paged_kv_cache_146_gb300 as P
from paged_kv_cache_146_gb300 import build


class Ran:
    returncode, stdout, stderr = 0, "", ""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() in an empty folder: compiling and linking only make their files."""
    for name in ("LIB", "FASTCALL"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "_compile", lambda src, *a: str(tmp_path / src))
    (tmp_path / "_fastcall.so").write_text("an earlier one")
    return tmp_path


def run_with(fail):
    def run(cmd, **kw):
        if cmd[0] == "g++":
            if fail == "missing":
                raise FileNotFoundError("g++")
            r = Ran()
            r.returncode, r.stderr = int(fail == "refuses"), "error: no such header"
            if not r.returncode:
                open(cmd[cmd.index("-o") + 1], "w").write("new")
            return r
        open(cmd[cmd.index("-o") + 1], "w").write("library")
        return Ran()
    return run


@pytest.mark.parametrize("fail", ["missing", "refuses"])
def test_the_library_is_built_without_a_compiler_for_the_checks(fail, tree, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(build.subprocess, "run", run_with(fail))
    monkeypatch.setattr(build.os.path, "exists", lambda p, real=os.path.exists: "include" in p or "lib" in p or real(p))
    with pytest.warns(UserWarning, match="_fastcall.so was not built"):
        lib = build.build()
    assert open(lib).read() == "library"
    assert sorted(os.listdir(tree)) == ["libpagedkv.so", "objects"]


def test_without_headers_an_earlier_module_goes(tree, monkeypatch):
    monkeypatch.setattr(build.subprocess, "run", run_with(None))
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    build.build()
    assert sorted(os.listdir(tree)) == ["libpagedkv.so", "objects"]


def test_a_checked_build_leaves_the_module_alone(tree, monkeypatch):
    monkeypatch.setattr(build.subprocess, "run", run_with(None))
    build.build(checked=True, out=str(tree / "checked.so"))
    assert (tree / "_fastcall.so").read_text() == "an earlier one"


@pytest.mark.parametrize("other", [{}, {"torch_version": "1.0"}, {"python_version": 207}, {"interface": "0"},
                                   {"interface": None}])
def test_a_module_made_for_something_else_is_not_taken(other, monkeypatch):
    torch = pytest.importorskip("torch")
    m = types.ModuleType(P.__name__ + "._fastcall")
    m.torch_version = torch.__version__.split("+")[0]
    m.python_version = sys.version_info[0] * 100 + sys.version_info[1]
    m.interface = build.interface_hash()
    for k, v in other.items():
        if v is None:
            delattr(m, k)                    # a module of before this attribute
        else:
            setattr(m, k, v)
    monkeypatch.setitem(sys.modules, m.__name__, m)
    monkeypatch.setattr(P, "_fastcall", m, raising=False)
    assert (P._load_fastcall(torch) is m) == (not other)


def test_the_interface_follows_the_header(tmp_path, monkeypatch):
    before = build.interface_hash()
    text = open(os.path.join(build.INCLUDE, "pagedkv.h")).read()
    (tmp_path / "pagedkv.h").write_text(text + "\n")
    monkeypatch.setattr(build, "INCLUDE", str(tmp_path))
    assert build.interface_hash() != before

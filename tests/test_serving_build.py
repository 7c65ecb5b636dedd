"""The compiled binding of the serving operators belongs to the torch that it was built
with, and the C libraries need neither torch nor Python's headers."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from rope_kv_cache_gb300 import _serving, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def test_the_binding_of_another_torch_is_not_loaded(monkeypatch):
    here = _serving._native().__file__
    assert os.path.exists(here)
    monkeypatch.setattr(_serving, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    with pytest.raises(RuntimeError, match="is not built"):
        _serving._native()
    compiled = []
    monkeypatch.setattr(build.subprocess, "Popen", lambda cmd, **kw: compiled.append(cmd) or _Failed())
    with pytest.raises(RuntimeError, match="ropekv_bind"):       # it would be built anew
        build.build_library()
    assert len(compiled) == 1 and build.BIND_SOURCE in compiled[0]
    monkeypatch.undo()
    assert _serving._native().__file__ == here


@pytest.mark.parametrize("lacks", ["torch", "Python.h", "a CUDA build of torch"])
def test_the_c_libraries_are_built_without_the_bindings_needs(monkeypatch, tmp_path, lacks):
    """Everything is stale; the compilers are stubs that write their output."""
    compiled = []

    def compiler(cmd, **kw):
        compiled.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return _Done()
    monkeypatch.setattr(build.subprocess, "Popen", compiler)
    monkeypatch.setattr(build.subprocess, "run", compiler)
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path))
    names = ("libropekv.so", "libropekv_floor.so", "libropekv_serving.so")
    for attr, n in zip(("LIB_PATH", "FLOOR_LIB_PATH", "SERVING_LIB_PATH"), names):
        monkeypatch.setattr(build, attr, str(tmp_path / n))
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif lacks == "Python.h":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setattr(torch, "__file__", str(tmp_path / "__init__.py"))
    with pytest.warns(UserWarning, match=lacks):
        assert build.build_library() == str(tmp_path / "libropekv.so")
    assert sorted(os.listdir(tmp_path)) == sorted(names)
    assert not any(build.BIND_SOURCE in c for c in compiled)


class _Done:
    returncode = 0

    def wait(self):
        return 0


class _Failed:
    def wait(self):
        return 1

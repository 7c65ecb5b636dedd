"""The compiled binding of the serving operators belongs to the torch that it was built
with, and the C libraries need neither torch nor Python's headers."""
import os

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


class _Failed:
    def wait(self):
        return 1

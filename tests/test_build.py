"""Building where PyTorch's binding cannot be built, or is another PyTorch's (CPU; no compiler runs)."""
import os
import shutil
import subprocess

import pytest

from bit_mla_kv_qdecode_b200 import _lib, api
from bit_mla_kv_qdecode_b200 import build as _build


@pytest.fixture
def built():
    _build.build()


@pytest.mark.parametrize("failure", ["no compiler", "no headers", "no toolkit"])
def test_the_library_stands_without_its_binding(built, monkeypatch, tmp_path, failure):
    binding = tmp_path / "_mla_torch.so"
    binding.write_bytes(b"of older sources")
    monkeypatch.setattr(_build, "binding_path", lambda: str(binding))
    monkeypatch.setattr(_build.os.path, "getmtime", lambda p, real=_build.os.path.getmtime: 0.0 if p == str(binding) else real(p))

    def run(cmd, **kw):
        if failure == "no compiler":
            raise FileNotFoundError(2, "No such file or directory", cmd[0])
        return subprocess.CompletedProcess(cmd, 1, "", "fatal error: cuda_runtime_api.h: No such file or directory")

    monkeypatch.setattr(_build.subprocess, "run", run)
    if failure == "no toolkit":
        def none():
            raise RuntimeError("nvcc not found")
        monkeypatch.setattr(_build, "nvcc_path", none)
    with pytest.warns(UserWarning, match="binding"):
        assert _build.build() == _build.LIB_PATH
    assert not binding.exists()  # not taken for a binding of this library
    assert _lib.load().mla_qcache_layout_version() == 1


def test_another_pytorch_has_another_binding(built, monkeypatch):
    import torch
    mine, ran = _lib.binding_path(), []
    assert os.path.exists(mine)

    def run(cmd, **kw):
        ran.append(cmd[cmd.index("-o") + 1])
        return subprocess.CompletedProcess(cmd, 1, "", "not run")

    monkeypatch.setattr(_build.subprocess, "run", run)
    _build.build()
    assert ran == []  # up to date
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert _lib.binding_path() != mine and not os.path.exists(_lib.binding_path())
    with pytest.warns(UserWarning, match="binding"):
        _build.build()
    assert len(ran) == 1 and ran[0].startswith(_lib.binding_path())
    assert os.path.exists(mine)


def test_a_missing_binding_is_built_on_import_when_asked_for(built, monkeypatch):
    mine = _build.binding_path()
    other = mine[:-len(".so")] + "-of-a-test.so"
    built_for = []
    monkeypatch.setattr(_build, "binding_path", lambda: other)
    monkeypatch.setattr(_build, "build_binding", lambda *a, **kw: (built_for.append(other), shutil.copy(mine, other)))
    monkeypatch.setattr(api, "_binding", None)
    monkeypatch.delenv("MLA_BUILD_ON_IMPORT", raising=False)
    with pytest.raises(ImportError, match="python -m"):
        api._ext()
    monkeypatch.setenv("MLA_BUILD_ON_IMPORT", "1")
    try:
        assert hasattr(api._ext(), "qdecode_sparse") and built_for == [other]
        monkeypatch.setattr(api, "_binding", None)
        api._ext()
        assert built_for == [other]  # it is there now
    finally:
        if os.path.exists(other):
            os.remove(other)

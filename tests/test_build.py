"""The build's functions (no GPU needed)."""
import os
import shutil

import pytest

from hyper_connection_residual_read_gb300 import build


@pytest.mark.parametrize("name", ["build_pycall", "build_pywindow"])
def test_call_modules_are_given_by_path_or_none(name, tmp_path, monkeypatch):
    monkeypatch.setattr(build, "PKG", os.fspath(tmp_path))
    path = getattr(build, name)()
    if shutil.which("gcc") or shutil.which("cc"):
        assert isinstance(path, str) and os.path.dirname(path) == os.fspath(tmp_path) and os.path.exists(path)
    monkeypatch.setattr(build.shutil, "which", lambda cc: None)
    assert getattr(build, name)() is None

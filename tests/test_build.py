"""What the build needs: the library nothing of Python's, the compiled part of
the binding the running Python and the installed torch."""
import importlib.metadata
import os
import sysconfig

import pytest

from discrete_selective_ssm_b200 import build


@pytest.fixture
def no_headers(monkeypatch):
    """A machine without Python.h and torch's C++ headers."""
    def fails(*_):
        raise OSError("no Python.h, no torch headers")
    monkeypatch.setattr(build, "build_bind", fails)
    monkeypatch.setattr(build, "_stale", lambda: False)  # (compiling is not what is tested)


def test_the_library_needs_no_python_headers(no_headers):
    assert build.build() == build.LIB


def test_a_binding_of_another_python_or_torch_is_not_taken(monkeypatch):
    path = build.bind_path()
    assert os.path.dirname(path) == build.HERE
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version",
                        lambda name: "0.0.1" if name == "torch" else version(name))
    other_torch = build.bind_path()
    var = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda name: "cpython-30-none" if name == "SOABI" else var(name))
    assert len({path, other_torch, build.bind_path()}) == 3

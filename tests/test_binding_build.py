"""The serving calls' native binding belongs to the torch and the Python that it was built against: with others the
Python binding serves alone, and build() makes one for them."""
import os
import shutil

import pytest
import torch

import bit_weight_only_w4a16_gb300 as w4
from bit_weight_only_w4a16_gb300 import build


def test_built_and_loaded():
    """Where it can be built it is there: the tests of it are not passed over unseen."""
    include = os.path.join(os.path.dirname(torch.__file__), "include", "ATen", "core", "Tensor.h")
    if shutil.which("g++") is None or not os.path.exists(include):
        pytest.skip("no compiler, or no headers of torch")
    assert build.build_binding() == build.binding_path()
    assert os.path.exists(build.binding_path())
    assert w4._fast is not None and os.path.samefile(w4._fast.__file__, build.binding_path())


@pytest.mark.parametrize("what", ["version", "git", "python"])
def test_another_torch_or_python(monkeypatch, what):
    """One built for another torch or Python is neither current nor loaded."""
    mine = build.binding_path()
    if what == "version":
        monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    elif what == "git":
        monkeypatch.setattr(torch.version, "git_version", "0123456789abcdef")
    else:
        real = build.sysconfig.get_config_var
        monkeypatch.setattr(build.sysconfig, "get_config_var", lambda n: ".cpython-30-x.so" if n == "EXT_SUFFIX" else real(n))
    assert build.binding_path() != mine
    assert not build.binding_current()
    assert w4._load_binding() is None


def test_an_object_that_does_not_load_is_left(monkeypatch, tmp_path):
    bad = tmp_path / "_binding.x.so"
    bad.write_bytes(b"not an object")
    monkeypatch.setattr(build, "binding_path", lambda: str(bad))
    assert w4._load_binding() is None

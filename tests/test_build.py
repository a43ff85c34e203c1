"""The build of the shared library and of the Python binding, on a directory of
tiny sources: libsf.so needs neither torch nor a binding that compiles."""

import ctypes
import importlib.util
import os
import sys

import pytest

from greedy_speculative_decoding_gb300 import build as B


TINY = 'extern "C" __attribute__((visibility("default"))) int sf_tiny() { return 7; }\n'


def load(tmp, binding):
    """The build module by itself, as `python build.py` runs it, on sources of its own in tmp."""
    spec = importlib.util.spec_from_file_location("build_alone", B.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    csrc = tmp / "csrc"
    csrc.mkdir()
    (csrc / "tiny.cu").write_text(TINY)
    (csrc / "paged_py.cpp").write_text(binding)
    mod.CSRC, mod.BUILD_DIR = str(csrc), str(tmp / "objects")
    mod.HERE, mod.OUT, mod.PY_OUT = str(tmp), str(tmp / "libsf.so"), str(tmp / "_paged.so")
    return mod


@pytest.fixture
def build(tmp_path):
    return lambda binding: load(tmp_path, binding)


def test_library_without_torch(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)   # an import of it fails
    mod = build("#error not compiled without torch\n")
    assert ctypes.CDLL(mod.build()).sf_tiny() == 7
    assert not os.path.exists(mod.PY_OUT)
    at = os.path.getmtime(mod.OUT)
    mod.build()
    assert os.path.getmtime(mod.OUT) == at            # nothing changed: not built again


def test_library_when_the_binding_does_not_compile(build):
    mod = build("#error no\n")
    with pytest.raises(RuntimeError, match="binding failed"):
        mod.build()
    assert os.path.exists(mod.OUT) and not os.path.exists(mod.PY_OUT)
    with pytest.raises(RuntimeError, match="binding failed"):
        mod.build()                          # and not taken for finished


def test_binding_beside_the_library(build):
    mod = build('extern "C" int sf_tiny(); extern "C" int twice() { return 2 * sf_tiny(); }\n')
    mod.build()
    assert os.path.exists(mod.OUT) and os.path.exists(mod.PY_OUT)


def test_a_kernel_source_that_does_not_compile(build):
    mod = build("int x;\n")
    with open(os.path.join(mod.CSRC, "bad.cu"), "w") as f:
        f.write("#error no\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        mod.build()
    assert not os.path.exists(mod.OUT)

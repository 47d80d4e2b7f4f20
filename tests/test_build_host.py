"""The build's host logic, on a library of one small source.  No GPU is used."""
import ctypes
import os
import sys

import pytest

from onnx_lstm_gru_gb300 import _build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A tree of its own: one source, no binding yet."""
    csrc, out = tmp_path / "csrc", tmp_path / "out"
    csrc.mkdir()
    (csrc / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "probe.cu").write_text('extern "C" int probe() { return 2; }\n')
    for name, value in (("CSRC", csrc), ("BUILD", out), ("LIB", out / "librk.so"), ("PROBE_SRC", tmp_path / "probe.cu"),
                        ("PROBE_LIB", out / "libprobe.so"), ("BINDING_LIB", out / "binding.so")):
        monkeypatch.setattr(_build, name, str(value))
    return tmp_path


def test_library_is_built_without_torch(small, monkeypatch):
    """A user of the C library needs no torch: only the module that packs
    torch's tensors is left out."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert ctypes.CDLL(_build.build()).one() == 1
    assert not os.path.exists(_build.BINDING_LIB)


def test_library_is_built_before_a_binding_that_fails(small, monkeypatch):
    (small / "bad.cpp").write_text("#error not today\n")
    monkeypatch.setattr(_build, "BINDING_SRC", str(small / "bad.cpp"))
    with pytest.raises(RuntimeError, match="not today"):
        _build.build()
    assert ctypes.CDLL(_build.LIB).one() == 1


def test_binding_follows_the_installed_torch(small, monkeypatch):
    """Another torch has other headers and another binary interface."""
    torch = small / "site" / "torch"
    torch.mkdir(parents=True)
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.delitem(sys.modules, "torch", raising=False)
    monkeypatch.syspath_prepend(str(small / "site"))
    (small / "binding.cpp").write_text("")
    monkeypatch.setattr(_build, "BINDING_SRC", str(small / "binding.cpp"))
    built = []

    def binding():
        built.append(1)
        open(_build.BINDING_LIB, "w").close()
    monkeypatch.setattr(_build, "_build_binding", binding)
    for _ in range(2):
        _build.build()
        assert len(built) == 1
    (torch / "version.py").write_text("__version__ = '2'\n")
    for _ in range(2):
        _build.build()
        assert len(built) == 2

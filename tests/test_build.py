"""The build: the C library needs nvcc alone; the binding, torch's headers, is
left out with a message where it cannot be had, and refused by another torch."""
import ctypes
import importlib.util
import os
import sys
import types

import pytest


@pytest.fixture
def small(monkeypatch, tmp_path):
    """The build module on one source file, installing into a folder of its own."""
    from attention_fa_fwd_04_gb300 import build
    monkeypatch.setattr(build, "SOURCES", ["fa_decode_noalloc.cu"])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfa_gb300.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_fa_bind.so"))
    monkeypatch.setattr(build, "BIND_STAMP", str(tmp_path / "_fa_bind.torch"), raising=False)
    return build


def test_without_torch(small, monkeypatch, capfd):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert small.build() == small.LIB and os.path.exists(small.LIB)
    assert not os.path.exists(small.BIND)
    assert "torch is not installed" in capfd.readouterr().err
    assert small.up_to_date()
    when = os.stat(small.LIB).st_mtime_ns
    small.build()  # nothing is left to do
    assert os.stat(small.LIB).st_mtime_ns == when


@pytest.mark.parametrize("compiler", ["false", "no-such-compiler"])
def test_binding_that_does_not_compile(small, monkeypatch, capfd, compiler):
    open(small.BIND, "w").close()  # an older one
    monkeypatch.setenv("CXX", compiler)
    assert small.build() == small.LIB and os.path.exists(small.LIB)
    assert not os.path.exists(small.BIND)
    assert "left out" in capfd.readouterr().err
    when = os.stat(small.LIB).st_mtime_ns
    small.build()  # the binding alone is tried again
    assert os.stat(small.LIB).st_mtime_ns == when
    assert "left out" in capfd.readouterr().err


def test_library_that_does_not_compile(small, monkeypatch):
    monkeypatch.setattr(small, "NVCC", "false")
    with pytest.raises(RuntimeError, match="fa_decode_noalloc.cu"):
        small.build()
    assert not os.path.exists(small.LIB)


def test_another_torch_builds_the_binding_again(small, monkeypatch):
    version = small._torch()[1]
    import torch
    assert version == str(torch.__version__)
    open(small.BIND, "w").close()
    with open(small.BIND_STAMP, "w") as f:
        f.write(version)
    assert small._bind_up_to_date(version)
    assert not small._bind_up_to_date(version + ".1")
    os.utime(small.BIND, (1, 1))  # older than its sources
    assert not small._bind_up_to_date(version)


def test_binding_of_another_torch_is_refused(monkeypatch):
    import attention_fa_fwd_04_gb300 as fa
    lib = types.SimpleNamespace(**{n: ctypes.CFUNCTYPE(None)(lambda: None) for n in fa.EXPORTS})
    monkeypatch.setattr(fa, "load", lambda: lib)
    monkeypatch.setattr(fa, "_native", None)
    for other in (types.SimpleNamespace(torch_version="1.0", bind=pytest.fail),
                  types.SimpleNamespace(bind=pytest.fail)):
        monkeypatch.setitem(sys.modules, fa.__name__ + "._fa_bind", other)
        monkeypatch.setattr(fa, "_fa_bind", other, raising=False)
        with pytest.raises(ImportError, match="built against torch"):
            fa._load_native()
        assert fa._native is None

"""The build of the library and of the Python module beside it (nvcc and the host
compiler, no GPU)."""
import ctypes
import os

import pytest

from paged_kv_attention_12_gb300 import _build, binding


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one function and a module beside it, in a folder of their own."""
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "module.cpp").write_text("int two() { return 2; }\n")
    out = tmp_path / "lib"
    monkeypatch.setattr(_build, "_sources", lambda: [str(tmp_path / "one.cu")])
    monkeypatch.setattr(_build, "LIB_PATH", str(out / "libone.so"))
    monkeypatch.setattr(_build, "NATIVE_PATH", str(out / "_native.so"))
    monkeypatch.setattr(_build, "NATIVE_ABI", str(out / "_native.abi"), raising=False)
    monkeypatch.setattr(_build, "NATIVE_SRC", str(tmp_path / "module.cpp"))
    return tmp_path


def build():
    return _build.build(lib_path=_build.LIB_PATH)


def test_the_library_does_without_the_module(small):
    """Where the module does not compile there is the library, a warning, and no module of
    older sources."""
    (small / "module.cpp").write_text("#include <no_such_header_of_anyone.h>\n")
    os.makedirs(small / "lib")
    (small / "lib" / "_native.so").write_text("of older sources")
    os.utime(small / "lib" / "_native.so", (0, 0))
    with pytest.warns(RuntimeWarning, match="no_such_header_of_anyone"):
        path = build()
    assert ctypes.CDLL(path).one() == 1
    assert not os.path.exists(_build.NATIVE_PATH)
    with pytest.warns(RuntimeWarning, match="_native.so was not built"):
        assert build() == path             # the library is there: the module is tried again
    (small / "module.cpp").write_text("int two() { return 2; }\n")
    assert build() == path and os.path.exists(_build.NATIVE_PATH)


def test_a_library_that_fails_still_raises(small):
    (small / "one.cu").write_text("no C++\n")
    with pytest.raises(RuntimeError, match="nvcc failed on one.cu"):
        build()


def test_calls_without_their_module_say_so(monkeypatch):
    monkeypatch.setattr(binding, "_native_module", None)
    monkeypatch.setattr(binding, "HERE", os.path.join(binding.HERE, "nowhere"))
    with pytest.raises(RuntimeError, match="build it first"):
        binding._native()


def test_a_module_of_another_torch_is_built_again(small, monkeypatch):
    """Times of files do not show a change of torch or of Python."""
    import torch
    path = build()
    built = os.stat(_build.NATIVE_PATH).st_mtime_ns
    assert build() == path and os.stat(_build.NATIVE_PATH).st_mtime_ns == built
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        build()
        again = os.stat(_build.NATIVE_PATH).st_mtime_ns
        assert again > built
    build()
    assert os.stat(_build.NATIVE_PATH).st_mtime_ns > again


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    import torch
    _build.build()
    monkeypatch.setattr(binding, "_native_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="another Python or torch"):
        binding._native()
    monkeypatch.undo()
    assert binding._native() is not None

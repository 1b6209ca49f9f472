"""The library's build and load where the native part of the binding cannot be had."""
import os
import sys

import pytest


@pytest.fixture
def B(monkeypatch, tmp_path):
    """The build module, on one small source and a folder of its own."""
    from paged_kv_cache_212_gb300 import build as B
    try:
        B.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    source = tmp_path / "one.cpp"
    source.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(B, "_sources", lambda: [str(source)])
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "native_lib", lambda: str(tmp_path / "native.so"))
    monkeypatch.setattr(B, "NATIVE_SRC", str(tmp_path / "native.cpp"))
    return B


@pytest.mark.parametrize("fault", ["does not compile", "no compiler", "no torch"])
def test_the_library_is_built_without_the_binding(B, monkeypatch, tmp_path, fault):
    (tmp_path / "native.cpp").write_text("#error not today\n")
    (tmp_path / "native.so").write_text("of an older source")
    os.utime(tmp_path / "native.so", (1, 1))
    if fault == "no compiler":
        run = B.subprocess.run

        def no_gxx(cmd, **kw):
            if cmd[0] == "g++":
                raise FileNotFoundError("g++")
            return run(cmd, **kw)
        monkeypatch.setattr(B.subprocess, "run", no_gxx)
    if fault == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)      # import torch: ImportError
    with pytest.warns(RuntimeWarning, match="binding"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(tmp_path / "native.so")
    t = os.path.getmtime(B.LIB)
    with pytest.warns(RuntimeWarning, match="binding"):      # the library is up to date, the binding still missing
        assert B.build() == B.LIB
    assert os.path.getmtime(B.LIB) == t
    import ctypes
    assert ctypes.CDLL(B.LIB).one() == 1


def test_a_library_that_does_not_compile_is_an_error(B, monkeypatch, tmp_path):
    (tmp_path / "one.cpp").write_text("#error not today\n")
    (tmp_path / "native.cpp").write_text("#error not today\n")
    with pytest.raises(RuntimeError, match="one.cpp"):
        B.build()


def test_a_binding_that_does_not_load_is_left_out(monkeypatch, tmp_path):
    import paged_kv_cache_212_gb300 as P
    bad = tmp_path / "_native.so"
    bad.write_bytes(b"no shared object")
    monkeypatch.setattr(P, "NATIVE_PATH", str(bad))
    with pytest.warns(RuntimeWarning, match="binding"):
        assert P._load_native(None) is None
    monkeypatch.setattr(P, "NATIVE_PATH", str(tmp_path / "absent.so"))
    assert P._load_native(None) is None


def test_the_binding_is_named_after_what_it_was_built_for():
    """Another Python, machine or torch looks for another file."""
    import sysconfig

    import torch

    import paged_kv_cache_212_gb300 as P
    from paged_kv_cache_212_gb300 import build as B
    name = os.path.basename(P.NATIVE_PATH)
    assert B.native_lib() == P.NATIVE_PATH
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))

"""libtv.so loads and serves without the C++ side of the binding, and that side
is used only where it fits: built for this torch and interpreter, and for the
library that was loaded.  Each case runs in an interpreter of its own, on a copy
of the package; none needs a GPU."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

from paged_kv_cache_376_b200 import _lib, build

PKG = "paged_kv_cache_376_b200"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture
def copy(tmp_path):
    """The package's Python files and libtv.so, without the C++ side."""
    dst = tmp_path / PKG
    dst.mkdir()
    for name in os.listdir(build.PKG):
        if name.endswith(".py") or name == "libtv.so":
            shutil.copy(os.path.join(build.PKG, name), dst / name)
    return dst


def _python(cwd, code):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], cwd=cwd,
                       capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": str(cwd)})
    assert r.returncode == 0, r.stderr[-2000:]


CALL = """
    import torch
    from paged_kv_cache_376_b200 import _lib
    lib = _lib.load()
    assert _lib._fast is None
    assert lib.tv_status_string(0) == b"TV_OK"
    # a serving operator says what is wrong as ever
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    try:
        _lib.tv_page_copy(x, x, i, i)
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("a CPU tensor went through")
"""


def test_the_library_loads_without_the_fast_side(copy):
    _python(copy.parent, CALL)


def test_a_fast_side_of_another_torch_is_left_alone(copy):
    """Built for another torch or interpreter it has another name; one that
    does not load (here: not a library at all) is passed over too."""
    src = build.fast_path()
    (copy / os.path.basename(src).replace("torch", "torch9.")).write_bytes(
        open(src, "rb").read())
    (copy / "_fastcall.so").write_bytes(open(src, "rb").read())
    _python(copy.parent, CALL)
    (copy / os.path.basename(src)).write_bytes(b"no library")
    _python(copy.parent, CALL)


def test_the_fast_side_serves_its_own_library_alone(copy, tmp_path):
    shutil.copy(build.fast_path(), copy)
    other = tmp_path / "other.so"
    shutil.copy(build.LIB_PATH, other)
    _python(copy.parent, """
        from paged_kv_cache_376_b200 import _lib
        _lib.load()
        assert _lib._fast.chunk
    """)
    _python(copy.parent, f"""
        from paged_kv_cache_376_b200 import _lib
        _lib.load({str(other)!r})
        assert _lib._fast is None
    """)


def test_a_missing_library_is_a_tv_error(copy):
    (copy / "libtv.so").unlink()
    _python(copy.parent, """
        from paged_kv_cache_376_b200 import _lib
        try:
            _lib.load()
        except _lib.TVError as e:
            assert "build it" in str(e)
        else:
            raise AssertionError
    """)


def test_the_name_goes_by_torch_and_interpreter(monkeypatch):
    import torch
    here = build.fast_path()
    assert os.path.exists(here)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert build.fast_path() != here


def test_the_fast_side_is_rebuilt_after_a_change_of_its_build(monkeypatch):
    assert build.fast_up_to_date()
    stamp = os.path.getmtime(build.fast_path())
    real = os.path.getmtime
    for name in ("build.py", os.path.join("csrc", "fastcall.cpp")):
        path = os.path.join(build.PKG, name)
        monkeypatch.setattr(os.path, "getmtime",
                            lambda p, path=path: stamp + 1 if p == path
                            else real(p))
        assert not build.fast_up_to_date()
    monkeypatch.undo()
    assert build.fast_up_to_date()
    assert _lib.LIB_PATH == build.LIB_PATH

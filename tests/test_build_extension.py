"""The Python extension of the hot calls is optional: whatever goes wrong with
it, libhs.so is built and loaded, and no extension of another build is used."""
import os
import warnings

import pytest

from sparse_top_kv_gb300 import _build, hs


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own."""
    src = tmp_path / "csrc"
    out = tmp_path / "out"
    src.mkdir()
    out.mkdir()
    (src / "hs_small.cu").write_text('extern "C" int hs_small() { return 7; }\n')
    (src / "hs_binding.cpp").write_text("#error not this time\n")
    monkeypatch.setattr(_build, "CSRC", str(src))
    monkeypatch.setattr(_build, "OUT_DIR", str(out))
    monkeypatch.setattr(_build, "LIB", str(out / "libhs.so"))
    return out


def need_compilers():
    if _build._python_include() is None:
        pytest.skip("no C++ compiler or no Python headers")
    try:
        _build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")


def test_library_without_the_extension(elsewhere, monkeypatch):
    need_compilers()
    (elsewhere / "_hs_binding-cpython-30-torch0.1.so").write_text("another Python's")
    path = _build.binding_path()
    open(path, "w").write("an older build's")
    os.utime(path, (1, 1))
    with pytest.warns(UserWarning, match="not this time"):
        assert _build.build() == str(elsewhere / "libhs.so")
    assert os.path.exists(elsewhere / "libhs.so")
    assert not [f for f in os.listdir(elsewhere) if f.startswith("_hs_binding") and f.endswith(".so")]
    with warnings.catch_warnings():  # not tried again as long as nothing changes
        warnings.simplefilter("error")
        monkeypatch.setattr(_build, "_gcc", lambda *a: pytest.fail("tried again"))
        _build.build()


def test_headers_gone_after_a_build(elsewhere, monkeypatch):
    need_compilers()
    monkeypatch.setattr(_build, "_python_include", lambda: None)
    (elsewhere / "_hs_binding-cpython-30-torch0.1.so").write_text("cannot be rebuilt")
    (elsewhere / "_hs_binding.so").write_text("an older name")
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _build.build()
    assert _build.binding_path() is None
    assert sorted(os.listdir(elsewhere)) == ["hs_small.o", "libhs.so"]


def test_name_tells_python_and_torch(monkeypatch):
    import torch
    if _build.binding_path() is None:
        pytest.skip("no C++ compiler or no Python headers")
    here = _build.binding_path()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert _build.binding_path() != here


def test_extension_that_does_not_load(tmp_path, monkeypatch):
    bad = tmp_path / "bad.so"
    bad.write_text("not a library")
    monkeypatch.setattr(hs, "_binding", None)
    monkeypatch.setattr(_build, "binding_path", lambda: str(bad))
    with pytest.warns(UserWarning, match="does not load"):
        hs._load_binding()
    assert hs._binding is None

"""What the build makes, without a compiler."""

import warnings

import pytest

from paged_kv_cache_page_gb300 import build as pabuild


def test_the_library_is_linked_where_the_python_module_cannot_be_built(monkeypatch, tmp_path):
    """The C library needs neither Python's headers nor torch's."""
    linked = []
    monkeypatch.setattr(pabuild, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(pabuild, "_compile", lambda src, obj, extra, verbose: open(obj, "w").close() or "")
    monkeypatch.setattr(pabuild, "_link", lambda lib, objs: linked.append(lib))

    def fails(lib, verbose):
        raise RuntimeError("Python.h: No such file or directory")

    monkeypatch.setattr(pabuild, "_build_binding", fails)
    stale = tmp_path / pabuild.BINDING_LIB
    stale.write_text("of older sources")
    with warnings.catch_warnings(record=True) as told:
        warnings.simplefilter("always")
        path = pabuild.build(force=True)
    assert path == pabuild.lib_path() and path in linked
    assert any("Python.h" in str(w.message) for w in told)
    assert not stale.exists()  # a module that does not fit the library is not left to be loaded
    # a kernel that does not compile still ends the build
    monkeypatch.setattr(pabuild, "_compile", fails_to_compile)
    with pytest.raises(RuntimeError, match="nvcc"):
        pabuild.build(force=True)


def fails_to_compile(src, obj, extra, verbose):
    raise RuntimeError("nvcc failed on " + src)

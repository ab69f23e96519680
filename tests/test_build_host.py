"""CPU checks of the build: the library does not depend on the binding's extension module."""
import os
import sysconfig

import pytest

import sharded_gemm_gb300 as tp
from sharded_gemm_gb300 import build as tpbuild


def test_library_builds_without_python_headers(tmp_path, monkeypatch, capfd):
    """Where Python.h is missing the library is built and loads; the functions that need the extension say so."""
    tpbuild.build()
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(tpbuild.sysconfig, "get_paths", lambda: paths)
    missing = str(tmp_path / os.path.basename(tpbuild.MARSHAL))
    monkeypatch.setattr(tpbuild, "MARSHAL", missing)
    assert tpbuild.build() == tpbuild.LIB and os.path.exists(tpbuild.LIB)
    assert not os.path.exists(missing)
    assert "Python.h" in capfd.readouterr().err
    assert tp.tp_version() > 0
    monkeypatch.setattr(tp, "MARSHAL_PATH", missing)
    monkeypatch.setattr(tp, "_native", None)
    with pytest.raises(RuntimeError, match="_marshal"):
        tp.tp_sample(None, None)


def test_an_extension_of_older_sources_is_not_left(tmp_path, monkeypatch):
    stale = tmp_path / os.path.basename(tpbuild.MARSHAL)
    stale.write_bytes(b"")
    os.utime(stale, (0, 0))
    monkeypatch.setattr(tpbuild.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(tpbuild, "MARSHAL", str(stale))
    assert tpbuild.build_marshal() is None
    assert not stale.exists()


def test_extension_is_named_for_its_interpreter():
    assert tpbuild.MARSHAL == tp.MARSHAL_PATH
    assert sysconfig.get_config_var("SOABI") in os.path.basename(tpbuild.MARSHAL)
    tpbuild.build()
    from sharded_gemm_gb300 import _marshal
    assert os.path.samefile(_marshal.__file__, tpbuild.MARSHAL)

"""The build's steps without a compiler: what is made where the extension module cannot be."""
import os
import stat

import pytest


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The build's products in an empty folder, and an nvcc that writes the file that it is asked for."""
    from autoregressive_decode_persistent_gb300 import build
    here = tmp_path / "package"
    here.mkdir()
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "adp.h").write_text("")
    for name in ("LIB", "TEST_LIB", "BINDING"):
        monkeypatch.setattr(build, name, str(here / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "FLAGS_STAMP", str(here / "_build" / "flags.txt"))
    monkeypatch.setattr(build, "HERE", str(here))
    fake = tmp_path / "nvcc"
    fake.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then : > "$2"; fi; shift; done\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "nvcc", lambda: str(fake))
    return build


def _fails():
    raise RuntimeError("Python.h: no such file")


def test_the_libraries_need_no_extension_module(elsewhere, monkeypatch):
    build = elsewhere
    monkeypatch.setattr(build, "_build_binding", _fails)
    with pytest.warns(RuntimeWarning, match="Python.h: no such file"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.TEST_LIB) and not os.path.exists(build.BINDING)
    assert not build._stale()  # they are not built again for the module's sake
    made = os.stat(build.LIB).st_mtime_ns
    with pytest.warns(RuntimeWarning):
        build.build()
    assert os.stat(build.LIB).st_mtime_ns == made


def test_a_module_of_other_sources_does_not_outlive_a_build_that_fails(elsewhere, monkeypatch):
    build = elsewhere
    with open(build.BINDING, "w"):
        pass
    monkeypatch.setattr(build, "_build_binding", _fails)
    with pytest.warns(RuntimeWarning):
        build.build(force=True)
    assert not os.path.exists(build.BINDING)


def test_a_pytorch_that_is_missing_is_said(elsewhere, monkeypatch):
    build = elsewhere
    monkeypatch.setitem(__import__("sys").modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="torch"):
        build.build()
    assert os.path.exists(build.LIB)

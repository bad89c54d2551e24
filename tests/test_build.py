"""The build's steps without a compiler: what is made where the extension module cannot be, and when that module is out of date."""
import os
import stat
import sysconfig

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
    for name in ("FLAGS_STAMP", "BINDING_STAMP"):
        monkeypatch.setattr(build, name, str(here / "_build" / (name + ".txt")), raising=False)
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


def test_a_module_made_for_another_pytorch_or_python_is_out_of_date(elsewhere, monkeypatch):
    import torch
    build = elsewhere

    def compiles(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w"):
            return build.subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiles)
    assert build._stale_binding()
    build.build()
    assert not build._stale_binding()
    assert build.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0")
        assert build._stale_binding() and not build._stale()
        build.build()
        assert not build._stale_binding()
    assert build._stale_binding()
    build.build()
    assert not build._stale_binding()
    os.remove(build.BINDING)
    assert build._stale_binding()


def test_a_module_made_for_another_pytorch_is_not_called(monkeypatch):
    import torch
    from autoregressive_decode_persistent_gb300 import build, ops
    build.build()
    assert ops._native() is not None
    monkeypatch.setattr(ops, "_binding", None)
    monkeypatch.setattr(ops, "_missing", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.raises(RuntimeError, match="1.0"):
        ops.paged_kv_append(*[None] * 10)

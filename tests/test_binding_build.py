"""The Python binding's own module: the file that a build leaves, and a build that fails."""
import os
import sysconfig

import pytest


@pytest.fixture()
def build():
    from paged_gqa_decode_06_gb300 import build as b
    if b.build_binding() is None:
        pytest.skip("torch's headers do not build here")
    return b


def test_a_binding_of_another_python_is_not_loaded(build, monkeypatch):
    """It is compiled against one interpreter's object layout: the file's name says which."""
    import paged_gqa_decode_06_gb300 as pkg
    assert os.path.exists(build.binding_path())
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda n: ".cpython-399-other.so" if n == "EXT_SUFFIX" else real(n))
    monkeypatch.setattr(pkg, "_quick_module", pkg._UNSET)
    assert not os.path.exists(build.binding_path())
    assert pkg._quick() is None


class Ran:
    """A compiler's answer."""

    def __init__(self, returncode):
        self.returncode, self.stderr = returncode, "no such header"


@pytest.fixture()
def elsewhere(build, monkeypatch, tmp_path):
    """Builds go to a folder of the test's own, with the binding of an earlier build."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    old = build.binding_path()
    with open(old, "w") as f:
        f.write("an earlier build's")
    return old


@pytest.mark.parametrize("where", ["replace", "makedirs", "remove"])
def test_a_binding_that_cannot_be_written_says_so(build, elsewhere, monkeypatch, where):
    """No right to write, a full disk: a warning, and calls take the Python way."""
    def refuse(*a, **kw):
        raise PermissionError("no right to write")
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **kw: Ran(0))
    monkeypatch.setattr(build.os, where, refuse)
    with pytest.warns(UserWarning, match="no right to write"):
        assert build.build_binding(force=True) is None


def test_a_binding_of_other_sources_is_not_left(build, elsewhere, monkeypatch):
    """Where the compiler fails, an earlier build's file does not stand in for it."""
    import paged_gqa_decode_06_gb300 as pkg
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **kw: Ran(1))
    with pytest.warns(UserWarning, match="no such header"):
        assert build.build_binding(force=True) is None
    assert not os.path.exists(elsewhere)
    monkeypatch.setattr(pkg, "_quick_module", pkg._UNSET)
    assert pkg._quick() is None


def test_a_build_does_not_lose_the_bindings_error(build, monkeypatch, tmp_path):
    """What build_binding does not expect reaches the caller of build()."""
    def broken(force=False):
        raise RuntimeError("not foreseen")
    monkeypatch.setattr(build, "build_binding", broken)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / build.LIB_NAME))
    monkeypatch.setattr(build, "_sources", lambda: [])
    monkeypatch.setattr(build, "_compile", lambda *a: ("", ""))
    with pytest.raises(RuntimeError, match="not foreseen"):
        build.build()

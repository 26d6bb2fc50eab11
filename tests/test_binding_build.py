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

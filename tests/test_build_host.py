"""When the native binding counts as up to date."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "quantized_mixture_experts_grouped_b200")


@pytest.fixture(scope="module")
def script():
    spec = importlib.util.spec_from_file_location("_moe_build_script", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_binding_is_built_again_for_another_torch(script, tmp_path, monkeypatch):
    """A module newer than its sources is stale all the same once torch, its C++ ABI or the interpreter
    has changed, or where nothing says what it was built for."""
    import sysconfig

    import torch
    so = tmp_path / "_rows.so"
    assert not script._binding_is_current(str(so))
    so.write_bytes(b"")
    assert not script._binding_is_current(str(so))                     # no stamp
    stamp = tmp_path / "_rows.so.stamp"
    stamp.write_text(script._binding_stamp())
    assert script._binding_is_current(str(so))
    os.utime(so, (1, 1))
    assert not script._binding_is_current(str(so))                     # older than its sources
    os.utime(so)
    for target, name, value in ((torch, "__version__", "0.0"), (torch._C, "_GLIBCXX_USE_CXX11_ABI",
                                                                not torch._C._GLIBCXX_USE_CXX11_ABI)):
        with monkeypatch.context() as m:
            m.setattr(target, name, value)
            assert not script._binding_is_current(str(so)), name
    with monkeypatch.context() as m:
        real = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda n: "cpython-00" if n == "SOABI" else real(n))
        assert not script._binding_is_current(str(so))
    assert script._binding_is_current(str(so))


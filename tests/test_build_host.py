"""When the native binding counts as up to date, and what works without it."""
import importlib.util
import os
import subprocess
import sys

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



@pytest.mark.parametrize("broken", ["sys.modules[name + '._rows'] = None",
                                    "import torch; torch.__version__ = '0.0.1+cpu'"])
def test_layer_calls_without_the_native_binding(broken):
    """Where _rows.so is missing or built for another torch, the package imports and the calls through
    ctypes work; a row operator's call raises and says what to do."""
    code = f"""
import sys
name = "quantized_mixture_experts_grouped_b200"
{broken}
import quantized_mixture_experts_grouped_b200 as q
assert q.moe_packed_bytes(256, 256) == 256 * 256 // 2 and q.moe_workspace_bytes(4, 256, 128, 8, 2) > 0
assert q.moe_norm_workspace_bytes(4, 8) > 0
try:
    q.moe_norm_pre(None, None, 1e-5, None)
except ImportError as e:
    assert "build.py" in str(e)
else:
    raise AssertionError("the call did not raise")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]

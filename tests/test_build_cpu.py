"""What needs what to build: the library stands without the extension."""
import subprocess
import sys
import textwrap

import pytest

from tests.conftest import ROOT


def _python(body):
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(body)], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("compiler", ["false", "/no/such/compiler"])
def test_the_int8_routes_load_without_the_extension(compiler, tmp_path):
    """No C++ compiler, or no headers of torch: the routes that go through ctypes work, the others say why not."""
    _python(f"""
        from w8a8_int8_quantized_i8_gb300 import build
        build.CALLS_LIB = {str(tmp_path / "_calls.so")!r}
        build._calls_compile = lambda obj: [{compiler!r}]
        import w8a8_int8_quantized_i8_gb300 as i8
        assert i8.load().i8_version() and i8.workspace_bytes(2560, 1024, 1024) >= 0
        for call in (build.build, i8.binding.load_calls, lambda: i8.quant_rows_fp4(None)):
            try:
                call()
            except RuntimeError as e:
                assert "_calls" in str(e), e
            else:
                raise AssertionError("built without a compiler")
        assert i8.load().i8_version()
    """)


def test_both_are_loaded_where_they_build():
    _python("""
        import w8a8_int8_quantized_i8_gb300 as i8
        assert i8.load() and i8.binding.load_calls() is i8.binding.load_calls()
        assert not i8.build.stale()
    """)


def test_an_extension_of_another_torch_or_python_is_not_taken():
    """After an upgrade the old binary lies there still, newer than its sources."""
    import importlib
    import sysconfig

    import torch

    from w8a8_int8_quantized_i8_gb300 import build
    names = {build.CALLS_LIB}
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1+other")
        names.add(importlib.reload(build).CALLS_LIB)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name, _f=sysconfig.get_config_var: "cpython-00-other" if name == "SOABI" else _f(name))
        names.add(importlib.reload(build).CALLS_LIB)
    assert len(names) == 3 and importlib.reload(build).CALLS_LIB in names

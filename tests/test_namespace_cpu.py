"""The package's namespace as its users see it: dir(), ``import *`` and attributes
hold every public binding of both modules, and nothing that a module only uses."""
import inspect
import subprocess
import sys

import pytest

import test_binding_streams_cpu
import test_layers_bindings_cpu
from conftest import ROOT


@pytest.fixture
def mx():
    from mlp_gemms_gb300 import build
    build.build()
    import mlp_gemms_gb300
    return mlp_gemms_gb300


def _public(module):
    return {n for n, f in vars(module).items()
            if n[0] != "_" and (inspect.isfunction(f) or inspect.isclass(f) or hasattr(f, "cache_info"))
            and f.__module__ == module.__name__}


def test_dir_and_star(mx):
    from mlp_gemms_gb300 import layers
    star = {}
    exec("from mlp_gemms_gb300 import *", star)
    for name in _public(layers) | _public(mx):
        assert name in dir(mx) and name in star and star[name] is getattr(mx, name), name
    assert {"E4M3", "ACT_SWIGLU", "SCORE_SIGMOID", "BF16", "STATUS"} <= set(star)


def test_what_the_module_uses_is_not_offered(mx):
    mx.NVFP4  # the layers are loaded
    for name in ("torch", "_rows", "_gpu", "_mx"):
        with pytest.raises(AttributeError):
            getattr(mx, name)


def test_every_binding_with_a_stream_is_in_a_list(mx):
    nothing = {"mx_grouped_gemm_wgrad_f32", "mx_mlp_fwd_bwd", "mx_get_device_status", "mx_selftest_bounded_wait"}
    takes = {n for n in dir(mx) if n.startswith("mx_") and inspect.isfunction(getattr(mx, n))
             and "stream" in inspect.signature(getattr(mx, n)).parameters}
    assert takes - nothing == set(test_binding_streams_cpu.CALLS) | set(test_layers_bindings_cpu.CALLS)


def test_the_package_itself_needs_no_torch():
    code = "import sys, mlp_gemms_gb300 as m; assert 'mx_moe_topk' in dir(m) and 'torch' not in sys.modules"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)

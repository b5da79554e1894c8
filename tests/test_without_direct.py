"""The library without the compiled module for its shortest calls (_direct):
everything still works, through ctypes."""
import os
import subprocess
import sys

import pytest
import torch

from fp8_block_scaled_04_amd import binding as b, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_loads_without_the_module():
    if not os.path.exists(build.LIB):
        build.build()
    code = ("import sys, warnings; sys.modules['fp8_block_scaled_04_amd._direct'] = None\n"  # importing it raises
            "from fp8_block_scaled_04_amd import binding as b\n"
            "with warnings.catch_warnings(record=True) as w:\n"
            "    warnings.simplefilter('always')\n"
            "    assert b.lib() is b.lib() and b._direct is None\n"
            "assert len(w) == 1 and '_direct' in str(w[0].message), w\n"
            "assert b.status_string(b.FP8G_OK) and b.fp8_gemm_workspace_bytes(64, 256, 1024) >= 0\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr


def test_module_has_a_host_compiler(monkeypatch):
    """g++ where there is one, else ROCm's compiler, which the library itself is built with."""
    monkeypatch.setenv("CXX", "my-c++ -m64")
    assert build.host_cxx() == ["my-c++", "-m64"]
    monkeypatch.delenv("CXX")
    monkeypatch.setattr(build.shutil, "which", lambda name: "/usr/bin/g++" if name == "g++" else None)
    assert build.host_cxx() == ["/usr/bin/g++"]
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert os.path.basename(build.host_cxx()[0]) == "clang++" and os.path.exists(build.host_cxx()[0])


@pytest.mark.gpu
def test_calls_without_the_module(monkeypatch):
    assert torch.cuda.is_available(), "this test needs a GPU"
    from test_gpu_direct import NAMES, arguments
    b.lib()
    results = []
    for without in (False, True):
        if without:
            monkeypatch.setattr(b, "_direct", None)
        for name in NAMES:
            a = arguments()[name]
            if name == "moe_route":
                b.fp8_moe_route(a[0], a[1], a[2], a[3], *a[4:9], expert_idx=a[9], weights=a[10])
            else:
                getattr(b, "fp8_" + name)(*a)
            torch.cuda.synchronize()
            results.append([t for t in a if isinstance(t, torch.Tensor)])
    for x, y in zip(results[:len(NAMES)], results[len(NAMES):]):
        assert all(torch.equal(p, q) for p, q in zip(x, y))
